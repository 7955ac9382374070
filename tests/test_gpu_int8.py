"""The 8-bit (W8A8) operators on the GPU against plain numpy forms.

Row encoders and the norm: the 8-bit values equal those of the stated fp32 steps
exactly, and the 64-bit mathematics within half a unit; scales within the
roundings counted below.  Product: each output within its three fp32 roundings
(float(sum), the product of the scales, their product) and the output's own."""
import numpy as np
import pytest
import torch

from tests import int8_ref as ref
from vector_quantization_codec_b200 import qamw

pytestmark = pytest.mark.gpu
DEV = "cuda"
T = {"bf16": torch.bfloat16, "f32": torch.float32}
U32, UBF16 = ref.U32, ref.UBF16


def f32(t):
    return t.detach().float().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def values(rows, d, kind, seed, scale=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, d)) * scale
    x[:, g.random(d) < 0.01] *= 20
    return torch.from_numpy(x.astype(np.float32)).to(T[kind]).to(DEV)


def chan_scale(d, seed):
    return torch.from_numpy(np.random.default_rng(seed).lognormal(0, 0.5, d).astype(np.float16)).to(DEV)


def check_rows(q, scale, h, c, s, gain, divide, eps=None):
    """q exactly; scale against 64 bits: v, a: <= 2 roundings, a / 127: 1 (encoders: <= 3).  The
    norm adds 1 / sqrt(sum / d + eps): the sum of squares of positive terms is off by at most one
    rounding per addition on a term's path, 32 in the thread, 10 in the two shuffle trees, and 1
    of the square; with / d and + eps 45, halved by the root, then root, reciprocal and product:
    23 + 3, in all <= 29."""
    hf = f32(h)
    q_want, scale_want, _ = ref.rows32(hf, c)
    np.testing.assert_array_equal(q.cpu().numpy(), q_want)
    got = scale.cpu().numpy().astype(np.float64)
    u64, scale64 = ref.rows64(hf, s, gain, divide, eps)
    n = 3 if eps is None else 29
    assert (np.abs(got - scale64) <= n * U32 * scale64 * (1 + 1e-6)).all()
    assert np.abs(q_want - u64).max() <= 0.5 + 5e-5
    if eps is None:
        np.testing.assert_array_equal(scale.cpu().numpy(), scale_want)


WIDTHS = [64, 128, 192, 512, 1024, 1088, 2048, 4096, 5120, 8192, 11008, 13824, 16448, 24640, 32768]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_encoders(d, kind):
    rows = 19
    x = values(rows, d, kind, d)
    x[rows - 1] = 0
    s = chan_scale(d, d + 1)
    for fn, divide, sc in ((qamw.qamw_int8_encode_weights, False, s),
                           (qamw.qamw_int8_encode_tokens, True, s),
                           (qamw.qamw_int8_encode_tokens, True, None)):
        st = status()
        q, scale = fn(x, sc, status=st)
        assert st.item() == 0
        sn = None if sc is None else sc.cpu().numpy()
        check_rows(q, scale, x, ref.factors32(d, sn, None, divide), sn, None, divide)
        assert scale[-1].item() == 0 and not q[-1].any()


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 149, 296, 297, 3001])
@pytest.mark.parametrize("d", [64, 1024, 2048])
def test_encoder_row_counts(rows, d):
    x = values(rows, d, "bf16", rows)
    q, scale = qamw.qamw_int8_encode_tokens(x)
    check_rows(q, scale, x, ref.factors32(d), None, None, True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", WIDTHS)
def test_rmsnorm(d, residual, kind):
    rows, eps = 13, 1e-5
    x = values(rows, d, kind, d)
    x[2] = 0
    res = values(rows, d, kind, d + 7, 3.0) if residual else None
    if residual:
        res[2] = 0
    gain = (1 + 0.2 * values(1, d, kind, 3)[0].clamp(-3, 3))
    for s in (None, chan_scale(d, 4)):
        st = status()
        out = qamw.qamw_rmsnorm_int8(x, gain, eps, residual=res, chan_scale=s, status=st)
        assert st.item() == 0
        h = x
        if residual:
            h, out = out[0], out[1:]
            assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
        sn = None if s is None else s.cpu().numpy()
        check_rows(*out, h, ref.factors32(d, sn, f32(gain), True), sn, f32(gain), True, eps)
        assert out[1][2].item() == 0 and not out[0][2].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [256, 1024, 1088, 2048, 4096, 5120, 6144, 8192, 11008, 12288, 13824, 16384,
                               16448, 25600, 32768])
def test_many_rows(d, kind):
    """Batches of more rows than the device takes at once, rows of zeros and of other scales among
    them."""
    rows, eps = 700, 1e-5
    x = values(rows, d, kind, d)
    x *= torch.logspace(-6, 4, rows, device=DEV).to(x.dtype)[:, None]
    x[[0, 311, rows - 1]] = 0
    s, sn = chan_scale(d, 4), chan_scale(d, 4).cpu().numpy()
    gain = (1 + 0.2 * values(1, d, kind, 3)[0].clamp(-3, 3))
    st = status()
    q, scale = qamw.qamw_int8_encode_weights(x, s, status=st)
    check_rows(q, scale, x, ref.factors32(d, sn, None, False), sn, None, False)
    for res in (None, x.flip(0).contiguous()):
        out = qamw.qamw_rmsnorm_int8(x, gain, eps, residual=res, chan_scale=s, status=st)
        h = x
        if res is not None:
            h, out = out[0], out[1:]
            assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
        check_rows(*out, h, ref.factors32(d, sn, f32(gain), True), sn, f32(gain), True, eps)
    assert st.item() == 0


@pytest.mark.parametrize("rows,d", [(1, 4096), (300, 64), (1000, 2048), (2, 32768), (999, 4096), (400, 32768)])
def test_rmsnorm_updates_the_residual_stream_in_place(rows, d):
    for alias in ("x", "residual"):
        x, res = values(rows, d, "bf16", 1), values(rows, d, "bf16", 2)
        gain = torch.ones(d, dtype=torch.bfloat16, device=DEV)
        want = qamw.qamw_rmsnorm_int8(x, gain, residual=res)
        got = qamw.qamw_rmsnorm_int8(x, gain, residual=res, sum_out=x if alias == "x" else res)
        assert got[0].data_ptr() == (x if alias == "x" else res).data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_with_nan_or_inf_are_flagged_and_stay_alone():
    for d in (256, 4096):
        x = values(6, d, "f32", 8)
        clean, _ = qamw.qamw_int8_encode_tokens(x)
        x[1, 3] = float("nan")
        x[4, d - 1] = -float("inf")
        for fn in (lambda st: qamw.qamw_int8_encode_tokens(x, status=st),
                   lambda st: qamw.qamw_int8_encode_weights(x, status=st),
                   lambda st: qamw.qamw_rmsnorm_int8(x, torch.ones(d, device=DEV), status=st)):
            st = status()
            q, scale = fn(st)
            assert st.item() == qamw.QAMW_STATUS_NONFINITE
            assert torch.isnan(scale).tolist() == [False, True, False, False, True, False]
            assert not q[1].any() and not q[4].any()
            keep = [0, 2, 3, 5]
            assert torch.equal(q[keep], clean[keep])
        # the product of such a token is NaN, and only that token's
        xq, xs = qamw.qamw_int8_encode_tokens(x)
        wq, ws = qamw.qamw_int8_encode_weights(values(70, d, "f32", 9))
        y = qamw.qamw_int8_gemm(xq, xs, wq, ws)
        assert torch.isnan(y).all(dim=1).tolist() == torch.isnan(xs).tolist()
        assert torch.isnan(y).any(dim=1).tolist() == torch.isnan(xs).tolist()


def test_extreme_magnitudes():
    """Rows near the ends of the range: values whose squares overflow or underflow, rows that are
    only just rows of zeros."""
    d, eps = 2048, 1e-6
    base = f32(values(1, d, "f32", 4))[0] / 100
    rows = np.stack([base * np.float32(v) for v in (1e37, 1e25, 1e18, 1.0, 1e-18, 1e-25, 2.0 ** -98)]
                    + [np.full(d, 2.0 ** -101, np.float32), np.full(d, 2.0 ** -100, np.float32)])
    x = torch.from_numpy(rows.astype(np.float32)).to(DEV)
    q, scale = qamw.qamw_int8_encode_tokens(x)
    q_want, scale_want, _ = ref.rows32(rows, ref.factors32(d))
    np.testing.assert_array_equal(q.cpu().numpy(), q_want)
    np.testing.assert_array_equal(scale.cpu().numpy(), scale_want)
    assert not q[7].any() and scale[7].item() == 0 and (q[8] == 127).all()
    st = status()
    q, scale = qamw.qamw_rmsnorm_int8(x, torch.ones(d, device=DEV), eps, status=st)
    assert st.item() == 0
    np.testing.assert_array_equal(q.cpu().numpy(), q_want)
    _, scale64 = ref.rows64(rows, None, None, True, eps)
    many = torch.cat([x] * 50)  # the same rows in a large batch
    for got_q, got_scale in (qamw.qamw_rmsnorm_int8(many, torch.ones(d, device=DEV), eps),
                             qamw.qamw_rmsnorm_int8(many, torch.ones(d, device=DEV), eps,
                                                    residual=torch.zeros_like(many))[1:]):
        assert torch.equal(got_q, q.repeat(50, 1))
        assert torch.allclose(got_scale, scale.repeat(50), rtol=64 * U32, atol=0)
    keep = [i for i in range(9) if i != 7]
    got = scale.cpu().numpy().astype(np.float64)
    # the rescaled sum of squares rounds three more times than the 29 of check_rows
    assert (np.abs(got - scale64) <= 32 * U32 * scale64 + 2.0 ** -149)[keep].all()


# ---------------------------------------------------------------- product

def ints(rows, d, seed, full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    return torch.randint(lo, 128, (rows, d), generator=g, dtype=torch.int8).to(DEV)


def scales(n, seed):
    return torch.from_numpy(np.random.default_rng(seed).lognormal(-3, 1, n).astype(np.float32)).to(DEV)


def check_gemm(xq, xs, wq, ws, dtype, y=None):
    st = status()
    got = qamw.qamw_int8_gemm(xq, xs, wq, ws, y=y, dtype=dtype, status=st)
    assert st.item() == 0, qamw.status_string(st.item())
    assert got.shape == (xq.shape[0], wq.shape[0]) and got.dtype == dtype
    a = xq.double() @ wq.double().T  # exact: |sum| <= 2^29
    want = a * (xs.double()[:, None] * ws.double()[None, :])
    tol = 3 * U32 + (UBF16 if dtype is torch.bfloat16 else 0)
    bad = (got.double() - want).abs() > tol * want.abs() * (1 + 1e-5)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())
    return got


TOKENS = [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 511, 1000]


@pytest.mark.parametrize("ntok", TOKENS)
def test_gemm_token_counts(ntok):
    for d_out, d_in in ((300, 1024), (129, 192), (328, 512), (200, 64)):
        check_gemm(ints(ntok, d_in, ntok), scales(ntok, 1), ints(d_out, d_in, 3), scales(d_out, 2),
                   torch.bfloat16)


@pytest.mark.parametrize("d_out", [1, 2, 7, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1001, 5003])
def test_gemm_output_widths(d_out):
    for ntok, d_in in ((1, 256), (6, 512), (40, 320), (140, 128), (300, 64)):
        check_gemm(ints(ntok, d_in, d_out), scales(ntok, 5), ints(d_out, d_in, 7), scales(d_out, 6),
                   torch.float32 if d_out % 2 else torch.bfloat16)


@pytest.mark.parametrize("d_in", [64, 128, 192, 256, 448, 1088, 4096, 4160, 11008, 13824, 32768])
def test_gemm_depths(d_in):
    for ntok, d_out in ((1, 130), (3, 64), (20, 200), (150, 300), (520, 260)):
        check_gemm(ints(ntok, d_in, 11), scales(ntok, 8), ints(d_out, d_in, d_in), scales(d_out, 9),
                   torch.float32)


@pytest.mark.parametrize("shape", [(1, 4096, 4096), (1, 11008, 4096), (7, 4096, 11008),
                                   (16, 4096, 11008), (64, 5120, 5120), (100, 4096, 11008),
                                   (333, 11008, 4096), (777, 13824, 5120), (2048, 4096, 4096)],
                         ids=str)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gemm_layer_shapes(shape, kind):
    ntok, d_out, d_in = shape
    check_gemm(ints(ntok, d_in, 1), scales(ntok, 2), ints(d_out, d_in, 3), scales(d_out, 4), T[kind])


@pytest.mark.parametrize("ntok", [290, 515, 777, 900, 1100, 2499])
def test_gemm_several_rounds_of_tiles(ntok):
    for d_out, d_in, kind in ((19000, 1024, "bf16"), (13824, 192, "bf16"), (19001, 320, "f32"), (5001, 2048, "bf16")):
        check_gemm(ints(ntok, d_in, ntok), scales(ntok, 1), ints(d_out, d_in, 5), scales(d_out, 2), T[kind])


@pytest.mark.parametrize("ntok", [1, 12, 100, 300])
def test_gemm_extreme_sums(ntok):
    """Sums of +-2^29 (all 256 values of int8 are allowed) and exact zeros."""
    d_in, d_out = 32768, 140
    for xv, wv in ((-128, -128), (-128, 127), (127, 127), (0, -128)):
        xq = torch.full((ntok, d_in), xv, dtype=torch.int8, device=DEV)
        wq = torch.full((d_out, d_in), wv, dtype=torch.int8, device=DEV)
        y = check_gemm(xq, torch.ones(ntok, device=DEV), wq, torch.ones(d_out, device=DEV), torch.float32)
        assert (y == float(xv * wv * d_in)).all()
    check_gemm(ints(ntok, d_in, 2, full=True), scales(ntok, 3), ints(d_out, d_in, 4, full=True),
               scales(d_out, 5), torch.bfloat16)


@pytest.mark.parametrize("ntok,d_out,kind", [(1, 77, "bf16"), (5, 77, "f32"), (13, 129, "bf16"),
                                             (70, 131, "bf16"), (130, 300, "f32"), (300, 257, "bf16")])
def test_gemm_writes_its_outputs_alone(ntok, d_out, kind):
    """y inside a larger buffer, at an odd element offset: what stands around it stays."""
    d_in, pad = 256, 1
    buf = torch.full((pad + ntok * d_out + 4096,), -7.0, dtype=T[kind], device=DEV)
    y = buf[pad:pad + ntok * d_out].view(ntok, d_out)
    check_gemm(ints(ntok, d_in, 1), scales(ntok, 2), ints(d_out, d_in, 3), scales(d_out, 4), T[kind], y)
    assert (buf[:pad] == -7).all() and (buf[pad + ntok * d_out:] == -7).all()


@pytest.mark.parametrize("ntok", [1, 9, 128, 400])
def test_gemm_is_the_same_every_time_and_reads_only_its_rows(ntok):
    d_in, d_out = 1024, 333
    big_x, big_w = ints(ntok + 300, d_in, 1), ints(d_out + 300, d_in, 2)
    xs, ws = scales(ntok + 300, 3), scales(d_out + 300, 4)
    want = qamw.qamw_int8_gemm(big_x[:ntok].clone(), xs[:ntok].clone(), big_w[:d_out].clone(),
                               ws[:d_out].clone())
    for _ in range(3):
        y = qamw.qamw_int8_gemm(big_x[:ntok], xs[:ntok], big_w[:d_out], ws[:d_out])
        assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """Inputs and outputs of more than 2^31 elements: the rows at the far end are those of a call
    on them alone."""
    d, rows = 32768, 70000
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
    tail = slice(rows - 300, rows)
    x.zero_()
    x[tail] = torch.randn((300, d), generator=g, device=DEV).to(torch.bfloat16)
    q, scale = qamw.qamw_int8_encode_tokens(x)
    q_tail, scale_tail = qamw.qamw_int8_encode_tokens(x[tail].clone())
    assert torch.equal(q[tail], q_tail) and torch.equal(scale[tail], scale_tail)
    assert not q[:300].any() and not scale[:300].any()
    h, qn, sn = qamw.qamw_rmsnorm_int8(x, torch.ones(d, dtype=torch.bfloat16, device=DEV), residual=x)
    hn, qt, st = qamw.qamw_rmsnorm_int8(x[tail].clone(), torch.ones(d, dtype=torch.bfloat16, device=DEV),
                                        residual=x[tail].clone())
    assert torch.equal(h[tail], hn) and torch.equal(qn[tail], qt) and torch.equal(sn[tail], st)
    del x, h, qn
    # as weights (more than 2^31 bytes), for a token and for many
    for ntok in (1, 3, 40, 300):
        xq, xs = ints(ntok, d, ntok), scales(ntok, 1)
        y = qamw.qamw_int8_gemm(xq, xs, q, scale, dtype=torch.float32)
        assert torch.equal(y[:, tail], qamw.qamw_int8_gemm(xq, xs, q_tail, scale_tail, dtype=torch.float32))
        assert not y[:, :1000].any()
    del q, y
    # outputs of more than 2^31 elements
    for kind in (torch.bfloat16, torch.float32):
        xq, xs, wq, ws = ints(65536, 64, 1), scales(65536, 2), ints(33000, 64, 3), scales(33000, 4)
        y = qamw.qamw_int8_gemm(xq, xs, wq, ws, dtype=kind)
        assert torch.equal(y[65000:], qamw.qamw_int8_gemm(xq[65000:], xs[65000:], wq, ws, dtype=kind))
        assert torch.equal(y[:300], qamw.qamw_int8_gemm(xq[:300], xs[:300], wq, ws, dtype=kind))
        del y


def test_products_on_several_streams_at_once():
    """CTAs, pairs and clusters that own tensor memory, and the codec's prefill product, all in
    flight together."""
    from tests.test_gpu_parity import codebook, gpu_encode, weights
    cb = codebook(7)
    Wt, _ = weights(512, 1024, 3, "bf16")
    m, _ = gpu_encode(Wt, 1024, 64, 7, cb, None, 0.0, seed=1)
    X = values(128, 1024, "bf16", 2)
    calls = [lambda: qamw.qamw_decode_gemm(m, X)]
    for ntok, d_out, d_in in ((300, 4096, 11008), (16, 4096, 11008), (1000, 4096, 1024), (1, 4096, 4096),
                              (64, 11008, 4096)):
        xq, xs, wq, ws = ints(ntok, d_in, 1), scales(ntok, 2), ints(d_out, d_in, 3), scales(d_out, 4)
        calls.append(lambda a=(xq, xs, wq, ws): qamw.qamw_int8_gemm(*a))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(12):
        for s, c, o in zip(streams, calls, got):
            with torch.cuda.stream(s):
                o.append(c())
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w, y) for y in o)


def test_empty_calls():
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    q, s = qamw.qamw_int8_encode_tokens(x)
    assert q.shape == (0, 128) and s.shape == (0,)
    h, q, s = qamw.qamw_rmsnorm_int8(x, torch.ones(128, dtype=torch.bfloat16, device=DEV), residual=x)
    assert h.shape == (0, 128) and q.shape == (0, 128)
    assert qamw.qamw_int8_gemm(q, s, ints(5, 128, 1), scales(5, 1)).shape == (0, 5)
    assert qamw.qamw_int8_gemm(ints(5, 128, 1), scales(5, 1), q, s).shape == (5, 0)


def test_wrappers_refuse_what_does_not_fit():
    x = values(4, 128, "bf16", 1)
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x.to(torch.float16))
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x[:, :64])                     # strided
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x, chan_scale(64, 1))          # too short
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x, chan_scale(128, 1).cpu())   # elsewhere
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x, chan_scale(128, 1).float())
    with pytest.raises(ValueError):
        qamw.qamw_int8_encode_tokens(x, q=torch.empty((3, 128), dtype=torch.int8, device=DEV))
    with pytest.raises(qamw.QamwError):
        qamw.qamw_int8_encode_tokens(values(4, 96, "bf16", 1))
    gain = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        qamw.qamw_rmsnorm_int8(x, gain.float())
    with pytest.raises(ValueError):
        qamw.qamw_rmsnorm_int8(x, gain, sum_out=x)
    with pytest.raises(ValueError):
        qamw.qamw_rmsnorm_int8(x, gain, residual=x[:2])
    with pytest.raises(qamw.QamwError):
        qamw.qamw_rmsnorm_int8(x, gain, eps=0.0)
    xq, xs, wq, ws = ints(4, 128, 1), scales(4, 1), ints(8, 128, 2), scales(8, 2)
    for bad in ((xq, xs, wq[:, :64], ws), (xq, xs[:3], wq, ws), (xq, xs, wq, ws.double()),
                (xq.to(torch.uint8), xs, wq, ws), (xq, xs, wq.cpu(), ws), (xq[0], xs, wq, ws)):
        with pytest.raises(ValueError):
            qamw.qamw_int8_gemm(*bad)
    with pytest.raises(ValueError):
        qamw.qamw_int8_gemm(xq, xs, wq, ws, dtype=torch.float16)
    with pytest.raises(ValueError):
        qamw.qamw_int8_gemm(xq, xs, wq, ws, y=torch.empty((4, 9), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        qamw.qamw_int8_gemm(xq, xs, wq, ws, status=torch.zeros(1, device=DEV))


# ---------------------------------------------------------------- together

def mlp(x, res, gain, wg, wu, wd, s_in, s_mid, status=None, stream=None):
    """Norm, gate and up projections, silu, down projection of a W8A8 layer."""
    h, q, ts = qamw.qamw_rmsnorm_int8(x, gain, residual=res, chan_scale=s_in, status=status, stream=stream)
    g = qamw.qamw_int8_gemm(q, ts, *wg, status=status, stream=stream)
    u = qamw.qamw_int8_gemm(q, ts, *wu, status=status, stream=stream)
    return h, g, u


def layer(d, f, ntok, seed):
    w = [values(f, d, "bf16", seed, 0.02), values(f, d, "bf16", seed + 1, 0.02),
         values(d, f, "bf16", seed + 2, 0.02)]
    s_in, s_mid = chan_scale(d, seed + 3), chan_scale(f, seed + 4)
    enc = [qamw.qamw_int8_encode_weights(w[0], s_in), qamw.qamw_int8_encode_weights(w[1], s_in),
           qamw.qamw_int8_encode_weights(w[2], s_mid)]
    x, res = values(ntok, d, "bf16", seed + 5), values(ntok, d, "bf16", seed + 6)
    gain = (1 + 0.1 * values(1, d, "bf16", seed + 7)[0].clamp(-3, 3))
    return w, enc, s_in, s_mid, x, res, gain


def full(x, res, gain, enc, s_in, s_mid):
    h, g, u = mlp(x, res, gain, enc[0], enc[1], enc[2], s_in, s_mid)
    a = torch.nn.functional.silu(g.float()) * u.float()
    q, ts = qamw.qamw_int8_encode_tokens(a.to(torch.bfloat16), s_mid)
    return h, a, q, ts, qamw.qamw_int8_gemm(q, ts, *enc[2])


def check_linear(y, n, W, q, ts, enc, s):
    """y against n W^T in 64 bits.  Each factor is off by at most half a unit of its row (and 5e-5
    for the fp32 roundings): with x' = n / s and W' = W s, |x' - ts q| <= 0.50005 ts and
    |W' - ws wq| <= 0.50005 ws, so |n W^T - product| <= 0.50005 (ts sum |W'| + ws sum |ts q|),
    plus the product's own roundings."""
    s, ts, wq, ws = s.double(), ts.double()[:, None], enc[0].double(), enc[1].double()[None, :]
    ys = ts * q.double() @ wq.T * ws
    off = 0.50005 * (ts * (W.double() * s).abs().sum(1)[None, :] + ws * (ts * q.double().abs()).sum(1)[:, None])
    want = n @ W.double().T
    assert ((y.double() - want).abs() <= off + 2 * (UBF16 + 3 * U32) * ys.abs()).all()


@pytest.mark.parametrize("ntok", [1, 3, 37, 200])
def test_mlp_of_a_w8a8_layer(ntok):
    """The operators one after another, as a layer uses them: norm, gate and up products, the
    activation encoded, down product; each product against the unquantised weights and inputs."""
    d, f = 512, 1408
    w, enc, s_in, s_mid, x, res, gain = layer(d, f, ntok, 20)
    h, q, ts = qamw.qamw_rmsnorm_int8(x, gain, residual=res, chan_scale=s_in)
    hd = (x.double() + res.double()).to(torch.bfloat16).double()
    assert torch.equal(h.double(), hd)
    n = hd * torch.rsqrt((hd * hd).mean(1, keepdim=True) + 1e-5) * gain.double()
    g, u = qamw.qamw_int8_gemm(q, ts, *enc[0]), qamw.qamw_int8_gemm(q, ts, *enc[1])
    check_linear(g, n, w[0], q, ts, enc[0], s_in)
    check_linear(u, n, w[1], q, ts, enc[1], s_in)
    a = (torch.nn.functional.silu(g.float()) * u.float()).to(torch.bfloat16)
    q, ts = qamw.qamw_int8_encode_tokens(a, s_mid)
    check_linear(qamw.qamw_int8_gemm(q, ts, *enc[2]), a.double(), w[2], q, ts, enc[2], s_mid)


def test_captured_graphs_and_streams():
    """Two captured graphs (which share nothing but their inputs) replayed in turn and on two
    streams at once give the eager results; so does a call on a stream that is not current."""
    d, f, ntok = 512, 1408, 5
    _, enc, s_in, s_mid, x, res, gain = layer(d, f, ntok, 40)
    want = full(x, res, gain, enc, s_in, s_mid)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            full(x, res, gain, enc, s_in, s_mid)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(full(x, res, gain, enc, s_in, s_mid))
        graphs.append(g)
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            t.zero_()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        h, g, u = mlp(x, res, gain, enc[0], enc[1], enc[2], s_in, s_mid, stream=stream)
        s.synchronize()
        assert torch.equal(h, want[0])
        h2, g2, u2 = mlp(x, res, gain, enc[0], enc[1], enc[2], s_in, s_mid)
        torch.cuda.synchronize()
        assert torch.equal(g, g2) and torch.equal(u, u2)


def test_inputs_freed_while_another_stream_still_reads_them():
    """Inputs dropped right after a call on a busy stream: their memory must not be handed to the
    next tensor of the current stream before the call has read it."""
    ntok, d, out = 64, 4096, 512
    wq, ws = ints(out, d, 1), scales(out, 2)
    x0 = values(ntok, d, "bf16", 3)
    q0, s0 = qamw.qamw_int8_encode_tokens(x0)
    y0 = qamw.qamw_int8_gemm(q0, s0, wq, ws)
    h0, n0, t0 = qamw.qamw_rmsnorm_int8(x0, torch.ones(d, dtype=torch.bfloat16, device=DEV), residual=x0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kind in ("tokens", "norm", "gemm"):
        a, b = (q0.clone(), s0.clone()) if kind == "gemm" else (x0.clone(), x0.clone())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        if kind == "tokens":
            got, want = qamw.qamw_int8_encode_tokens(a, stream=side), (q0, s0)
        elif kind == "norm":
            gain = torch.ones(d, dtype=torch.bfloat16, device=DEV)
            side.wait_stream(torch.cuda.current_stream())
            got, want = qamw.qamw_rmsnorm_int8(a, gain, residual=b, stream=side), (h0, n0, t0)
            del gain
        else:
            got, want = (qamw.qamw_int8_gemm(a, b, wq, ws, stream=side.cuda_stream),), (y0,)
        del a, b
        junk = [torch.full((ntok, d), 1, dtype=t, device=DEV) for t in (torch.bfloat16, torch.int8) * 3]
        junk += [torch.full((n,), 7.0, device=DEV) for n in (ntok, d, d // 2)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        del junk


def test_new_inputs_in_a_captured_graph():
    """A replay reads what its inputs hold then: other tokens, other weights."""
    xq, xs, wq, ws = ints(3, 512, 1), scales(3, 1), ints(200, 512, 2), scales(200, 2)
    y = torch.empty((3, 200), device=DEV)
    qamw.qamw_int8_gemm(xq, xs, wq, ws, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qamw.qamw_int8_gemm(xq, xs, wq, ws, y=y)
    for seed in (5, 6):
        xq.copy_(ints(3, 512, seed))
        wq.copy_(ints(200, 512, seed + 10))
        xs.copy_(scales(3, seed))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, check_gemm(xq, xs, wq, ws, torch.float32))


@pytest.mark.parametrize("ntok", [1, 2, 4, 16, 40, 300])
@pytest.mark.parametrize("d,out", [(256, 64), (2048, 1024), (4096, 4096)])
def test_buffers_rewritten_back_to_back(d, out, ntok):
    """Weights and tokens encoded into the same buffers again and again, each time followed at once
    by the product that reads them (every kernel launched before the one ahead ends): each product
    is that of its own step's values, neither older nor newer ones."""
    steps = 6
    W = [values(out, d, "bf16", 10 + i, 0.02) for i in range(steps)]
    X = [values(ntok, d, "bf16", 50 + i) for i in range(steps)]
    gain = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    want = []
    for w, x in zip(W, X):
        a, b = qamw.qamw_int8_encode_weights(w), qamw.qamw_rmsnorm_int8(x, gain)
        torch.cuda.synchronize()
        want.append(qamw.qamw_int8_gemm(*b, *a))
        torch.cuda.synchronize()
    wq, ws = torch.zeros((out, d), dtype=torch.int8, device=DEV), torch.zeros(out, device=DEV)
    xq, xs = torch.zeros((ntok, d), dtype=torch.int8, device=DEV), torch.zeros(ntok, device=DEV)
    y = [torch.zeros_like(want[0]) for _ in range(4 * steps)]
    torch.cuda.synchronize()
    for k, o in enumerate(y):
        qamw.qamw_rmsnorm_int8(X[k % steps], gain, q=xq, tok_scale=xs)
        qamw.qamw_int8_encode_weights(W[k % steps], q=wq, row_scale=ws)
        qamw.qamw_int8_gemm(xq, xs, wq, ws, y=o)
    torch.cuda.synchronize()
    for k, o in enumerate(y):
        assert torch.equal(o, want[k % steps]), k
    # captured: launches closer together still, tokens last
    def step(k):
        qamw.qamw_int8_encode_weights(W[k], q=wq, row_scale=ws)
        qamw.qamw_rmsnorm_int8(X[k], gain, q=xq, tok_scale=xs)
        qamw.qamw_int8_gemm(xq, xs, wq, ws, y=y[k])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for k in range(steps):
            step(k)
    for _ in range(3):
        for o in y:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for k in range(steps):
            assert torch.equal(y[k], want[k]), k


def test_product_feeds_the_decode_products():
    """In one stream with the codec's own kernels, each launched before the one ahead ends: the
    8-bit product's output as the input of a decode-GEMV and of the prefill product."""
    from tests.test_gpu_parity import codebook, gpu_encode, weights
    d, bits = 512, 7
    cb = codebook(bits)
    Wt, _ = weights(96, d, 3, "bf16")
    m, st = gpu_encode(Wt, d, 64, bits, cb, None, 0.0, seed=1)
    assert st == 0
    for ntok in (1, 4, 64):
        xq, xs, wq, ws = ints(ntok, 1024, 1), scales(ntok, 1), ints(d, 1024, 2), scales(d, 2)
        product = qamw.qamw_decode_gemv if ntok <= 16 else qamw.qamw_decode_gemm
        y = qamw.qamw_int8_gemm(xq, xs, wq, ws)
        torch.cuda.synchronize()
        want = product(m, y)
        torch.cuda.synchronize()
        out = torch.zeros_like(y)
        for _ in range(20):
            out.zero_()
            got = product(m, qamw.qamw_int8_gemm(xq, xs, wq, ws, y=out))
            q, _ = qamw.qamw_int8_encode_tokens(got.repeat(1, 2)[:, :128].contiguous())
            torch.cuda.synchronize()
            assert torch.equal(got, want)


@pytest.mark.parametrize("stage", ["int8_encode", "int8_norm", "int8_gemm"])
def test_benchmark_stage(stage, capsys):
    import json

    import bench
    assert bench.main(["--only", stage, "--rows", "384", "--din", "256", "--batch", "20", "--steps", "6",
                       "--warmup", "3"]) == 0
    line = json.loads(capsys.readouterr().out)
    assert line["stage"] == stage and line["ms"] > 0 and line["GB_per_s"] > 0
