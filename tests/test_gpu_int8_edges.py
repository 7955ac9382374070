"""The 8-bit (W8A8) operators where they are easily wrong: waits that give up, buffers that the
call ahead has just written, the ends of the range, first calls from several host threads."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import int8_ref as ref
from tests.test_gpu_int8 import DEV, T, check_gemm, ints, scales, status, values
from vector_quantization_codec_b200 import qamw

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ waits that give up

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,d", [(700, 1024), (300, 4096), (1000, 640), (450, 13312)])
def test_rows_after_a_wait_that_gives_up(rows, d, residual, kind):
    """A batch whose waits for rows give up at once, or after a few polls: flagged, and every CTA
    stops at a row: codes and scales are those of the whole call, or untouched.  The next call is
    not affected."""
    x = values(rows, d, kind, 1)
    res = values(rows, d, kind, 2) if residual else None
    gain = (1 + 0.2 * values(1, d, kind, 3)[0].clamp(-3, 3))
    want = qamw.qamw_rmsnorm_int8(x, gain, residual=res)
    for tries in (0, 0, 1, 2, 8, 64):
        q = torch.full((rows, d), -128, dtype=torch.int8, device=DEV)  # no row gives -128
        scale = torch.full((rows,), -1.0, device=DEV)
        h = res.clone() if residual else None  # the stream, updated in place
        st = status()
        qamw.qamw_selftest_rmsnorm_int8(tries, x, gain, h, q, scale, st, residual=h)
        torch.cuda.synchronize()
        done = scale >= 0
        assert st.item() == (0 if done.all() else qamw.QAMW_STATUS_TIMEOUT)
        assert torch.equal(q[done], want[-2][done]) and torch.equal(scale[done], want[-1][done])
        assert (q[~done] == -128).all() and (scale[~done] == -1).all()
        if residual:
            assert torch.equal(h[done], want[0][done])
            assert ((h == res) | (h == want[0])).all()
        if tries == 0:
            assert not done.any() and (h is None or torch.equal(h, res))
        st = status()
        again = qamw.qamw_rmsnorm_int8(x, gain, residual=res, status=st)
        assert st.item() == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


# ------------------------------------------------------------ data of the call ahead

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [576, 1024, 4096])
@pytest.mark.parametrize("ntok", [300, 1000])
def test_rows_read_what_the_call_ahead_has_just_written(ntok, d, kind):
    """A chain in which each call reads buffers that the call ahead has just rewritten with other
    values: a product's outputs as x of a norm, the norm's sum as the residual of the next, its
    codes as tokens of a product."""
    steps = 5
    gain = (1 + 0.2 * values(1, d, kind, 3)[0].clamp(-3, 3))
    w = [qamw.qamw_int8_encode_weights(values(d, d, kind, 20 + i, 0.1)) for i in range(steps)]
    x0 = values(ntok, d, kind, 1)
    y, h = torch.zeros((ntok, d), dtype=T[kind], device=DEV), torch.zeros((ntok, d), dtype=T[kind], device=DEV)
    q = torch.zeros((ntok, d), dtype=torch.int8, device=DEV)
    scale = torch.zeros(ntok, device=DEV)
    out = [[torch.zeros_like(t) for t in (y, h, q, scale)] for _ in range(steps)]

    def chain(wait, keep):
        h.copy_(x0)
        qamw.qamw_int8_encode_tokens(h, q=q, tok_scale=scale)
        for k in range(steps):
            wait()
            qamw.qamw_int8_gemm(q, scale, *w[k], y=y)
            wait()
            qamw.qamw_rmsnorm_int8(y, gain, residual=h, sum_out=h, q=q, tok_scale=scale)
            wait()
            qamw.qamw_rmsnorm_int8(h, gain, residual=h, sum_out=h, q=q, tok_scale=scale)
            if keep:
                wait()
                for a, b in zip(out[k], (y, h, q, scale)):
                    a.copy_(b)

    chain(torch.cuda.synchronize, True)  # nothing overlaps
    torch.cuda.synchronize()
    for _ in range(5):
        for t in (y, h, q, scale):
            t.zero_()
        chain(lambda: None, False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out[-1], (y, h, q, scale)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(lambda: None, False)
    for _ in range(5):
        for t in (y, h, q, scale):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out[-1], (y, h, q, scale)))


@pytest.mark.parametrize("many", [False, True])
def test_channel_scales_of_a_statistic_that_the_call_ahead_has_just_written(many):
    """Largest magnitudes per channel from the row encoder (x transposed: one row per channel),
    read at once by the channel scales: each step's scales are those of its own statistic."""
    d_in, ntok, steps, bits = 4096, 8192, 4, 6
    X = [values(d_in, ntok, "bf16", 70 + i, 1.0 + i) * (1 + torch.arange(d_in, device=DEV) % (5 + i))[:, None]
         for i in range(steps)]
    q, stat = torch.empty((d_in, ntok), dtype=torch.int8, device=DEV), torch.ones(d_in, device=DEV)
    cb = torch.randn((1 << bits, 2), device=DEV)
    W = values(64, d_in, "bf16", 5, 0.02)
    m = qamw.EncodedMatrix.empty(64, d_in, 64, bits, cb)
    ws = torch.empty(max(16, qamw.qamw_calibrate_many_workspace_bytes([m])), dtype=torch.uint8, device=DEV)

    def scales_of(k):
        qamw.qamw_int8_encode_tokens(X[k], q=q, tok_scale=stat)
        if many:
            qamw.qamw_calibrate_many([W], [m], [stat], 0.5, workspace=ws)
            return m.chan_scale.clone()
        return qamw.qamw_channel_scales(d_in, stat, 0.5, torch.empty(d_in, dtype=torch.float16, device=DEV))

    want = []
    for k in range(steps):
        qamw.qamw_int8_encode_tokens(X[k], q=q, tok_scale=stat)
        torch.cuda.synchronize()
        r = stat.double() / stat.double().mean()
        want.append(r.sqrt())
    for _ in range(3):
        got = [scales_of(k) for k in range(steps)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            # binary16 of the power: half a step, or half of the smallest step
            assert ((g.double() - w).abs() <= w * 2.0 ** -11 * (1 + 1e-6) + 2.0 ** -25).all()


# ------------------------------------------------------------ ends of the range

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 512, 2048, 8192, 13312, 28672, 32768])
def test_norm_of_rows_whose_squares_overflow(d, kind):
    """Rows of up to the type's largest value, whose sum of squares leaves binary32 by little or by
    far, with factors that bring the values back into range or near its other end."""
    largest = torch.finfo(T[kind]).max
    g = torch.Generator().manual_seed(d)
    u = torch.rand((6, d), generator=g) * 0.5 + 0.5
    u[:, ::3] *= -1
    rows = torch.stack([torch.full((d,), largest), u[0] * largest, u[1] * 3e38, u[2] * 1.5e38, u[3] * 2e19,
                        u[4] * 1e25, torch.where(torch.arange(d) == d // 2, 1e20, 1e-3)])
    x = rows.to(T[kind]).to(DEV)
    eps = 1e-5
    for factor, sc in ((1.0, None), (2.0 ** -60, 2.0 ** 4), (2.0 ** -100, 2.0 ** 14)):
        gain = torch.full((d,), factor, dtype=T[kind], device=DEV)
        s = None if sc is None else torch.full((d,), sc, dtype=torch.float16, device=DEV)
        sn = None if s is None else s.cpu().numpy()
        c = ref.factors32(d, sn, gain.float().cpu().numpy())
        xn = x.float().cpu().numpy()
        q_want, _, a = ref.rows32(xn, c)
        _, scale64 = ref.rows64(xn, sn, gain.float().cpu().numpy(), True, eps)
        many = x.repeat(50, 1)  # more rows than are taken one per CTA
        for got in (qamw.qamw_rmsnorm_int8(x, gain, eps, chan_scale=s),
                    qamw.qamw_rmsnorm_int8(x, gain, eps, residual=torch.zeros_like(x), chan_scale=s)[1:],
                    qamw.qamw_rmsnorm_int8(many, gain, eps, chan_scale=s),
                    qamw.qamw_rmsnorm_int8(many, gain, eps, residual=torch.zeros_like(many), chan_scale=s)[1:]):
            n = len(got[1]) // len(x)
            np.testing.assert_array_equal(got[0].cpu().numpy(), np.tile(q_want, (n, 1)))
            # v, a and a / 127: 3 roundings.  1 / rms: a sum of positive terms, each off by at most
            # one rounding per addition on its path (2 per 64 columns of a lane, 5 in the shuffles)
            # and the squares by one, halved by the root; then at most five more, and half of the
            # smallest step where the scale is that small
            tol = (3 + (2 * d / 64 + 5 + 1) / 2 + 5) * ref.U32
            want = np.tile(scale64 * (a >= ref.TINY), n)
            assert (np.abs(got[1].cpu().numpy() - want) <= tol * want + 2.0 ** -150).all()


# ------------------------------------------------------------ several host threads

FIRST_CALLS = """
import threading
import torch
from vector_quantization_codec_b200 import qamw

torch.manual_seed(0)
dev = "cuda"
ints = lambda r, d: torch.randint(-127, 128, (r, d), dtype=torch.int8, device=dev)
jobs = []  # per kernel, calls that need shared memory of different sizes, above 48 KB all
for t in (torch.bfloat16, torch.float32):
    for ntok in (1, 2):
        jobs.append([lambda a=(ints(ntok, d), torch.ones(ntok, device=dev), ints(64, d), torch.ones(64, device=dev)),
                     t=t: (qamw.qamw_int8_gemm(*a, dtype=t),) for d in (32768, 28672, 24576, 20480)])
    for norm in (False, True):
        for d in ((16448, 20480, 24576, 32768), (11008, 10240, 9216, 8192)):
            jobs.append([lambda x=torch.randn((400, w), device=dev).to(t), g=torch.ones(w, device=dev).to(t), norm=norm:
                         qamw.qamw_rmsnorm_int8(x, g) if norm else qamw.qamw_int8_encode_tokens(x) for w in d])
streams = [torch.cuda.Stream() for _ in range(8)]
torch.cuda.synchronize()
bad = []
for job in jobs:
    first, gate = {}, threading.Barrier(2 * len(job))
    def call(i):
        with torch.cuda.stream(streams[i]):
            gate.wait()
            try:
                first[i] = job[i % len(job)]()
            except qamw.QamwError as e:
                bad.append(str(e))
    threads = [threading.Thread(target=call, args=(i,)) for i in range(2 * len(job))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(2 * len(job)):
        try:
            again = job[i % len(job)]()
        except qamw.QamwError as e:
            bad.append(str(e))
            continue
        torch.cuda.synchronize()
        if i in first and not all(torch.equal(a, b) for a, b in zip(first[i], again)):
            bad.append("results differ")
assert not bad, bad
"""


def test_first_calls_of_several_host_threads():
    """Threads that make a kernel's first calls at the same time, with sizes that need different
    amounts of shared memory: none is refused, then or later, and all give the same results again."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):  # a new process each: what a call sets up lives as long as it
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------ kernels of a few tokens

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d_out,d_in", [(7104, 1024), (7105, 1024), (7200, 256), (7201, 448), (9003, 512), (7105, 2048),
                                        (7300, 2112), (4736, 4160), (4737, 4160), (8192, 4160), (11008, 5376),
                                        (11001, 5440), (3552, 6144), (3553, 6144), (3552, 32768), (3553, 32768),
                                        (5000, 26048), (65, 5632)])
def test_products_of_a_few_tokens_on_both_sides_of_each_rule(d_out, d_in, kind):
    """One to nine tokens where the choice of a kernel changes with the number of rows and their
    length: the exact sums, and a token's outputs the same bit for bit whatever comes with it."""
    x, w, xs, ws = ints(9, d_in, 1, full=True), ints(d_out, d_in, 2, full=True), scales(9, 3), scales(d_out, 4)
    want = check_gemm(x, xs, w, ws, T[kind])
    for ntok in (1, 2, 3, 5, 8):
        got = check_gemm(x[:ntok].contiguous(), xs[:ntok].contiguous(), w, ws, T[kind])
        assert torch.equal(got, want[:ntok])


@pytest.mark.parametrize("ntok,d_out,d_in", [(9, 2048, 4096), (16, 2047, 8192), (32, 2048, 2048), (12, 1900, 20480),
                                             (64, 2500, 8192), (40, 1000, 4096), (16, 4700, 11008)])
def test_products_whose_depth_clusters_share(ntok, d_out, d_in):
    """Few tiles: clusters of two to eight CTAs share a tile's depth, in one wave or more."""
    for kind in ("bf16", "f32"):
        check_gemm(ints(ntok, d_in, 1, full=True), scales(ntok, 2), ints(d_out, d_in, 3, full=True),
                   scales(d_out, 4), T[kind])


def test_checks_of_giving_up_refuse_what_does_not_fit():
    x, gain = values(4, 128, "bf16", 1), torch.ones(128, dtype=torch.bfloat16, device=DEV)
    q, scale, st = torch.empty((4, 128), dtype=torch.int8, device=DEV), torch.empty(4, device=DEV), status()
    norm = qamw.qamw_selftest_rmsnorm_int8
    for bad in ((x, gain[:64], None, q, scale, st), (x, gain, None, q[:3], scale, st), (x, gain, None, q, scale[:3], st),
                (x, gain, None, q, scale, st.cpu()), (x[:, :64], gain[:64], None, q, scale, st), (x, gain, x, q, scale, st)):
        with pytest.raises(ValueError):
            norm(0, *bad)
    with pytest.raises(ValueError):
        norm(0, x, gain, x[:2], q, scale, st, residual=x)
    w, y = ints(8, 128, 2), torch.empty((4, 8), device=DEV)
    for bad in ((q, scale, w[:, :64], scales(8, 1), y, st), (q, scale[:3], w, scales(8, 1), y, st),
                (q, scale, w, scales(7, 1), y, st), (q, scale, w, scales(8, 1), y[:3], st),
                (q, scale, w, scales(8, 1), y.half(), st), (q, scale, w, scales(8, 1), y, st.float())):
        with pytest.raises(ValueError):
            qamw.qamw_selftest_int8_gemm(*bad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm(64, x, gain, None, q, scale, st, stream=side)
    side.synchronize()
    want = qamw.qamw_rmsnorm_int8(x, gain)
    assert st.item() == 0 and torch.equal(q, want[0]) and torch.equal(scale, want[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ntok,d_out,d_in", [(100, 256, 256), (16, 4096, 11008), (64, 2048, 4096), (200, 4096, 4096),
                                             (300, 4096, 11008), (777, 5120, 2048), (2048, 9003, 1024)])
def test_products_whose_waits_give_up(ntok, d_out, d_in, kind):
    """Single CTAs, pairs and clusters whose roles give up at once: flagged, nothing written around
    the outputs, and the calls after it (which need its tensor memory) are not affected."""
    x, w, xs, ws = ints(ntok, d_in, 1), ints(d_out, d_in, 2), scales(ntok, 3), scales(d_out, 4)
    want = check_gemm(x, xs, w, ws, T[kind])
    buf = torch.full((ntok * d_out + 4096,), -7.0, dtype=T[kind], device=DEV)
    y = buf[2048:2048 + ntok * d_out].view(ntok, d_out)
    for _ in range(2):
        st = status()
        qamw.qamw_selftest_int8_gemm(x, xs, w, ws, y, st)
        got = qamw.qamw_int8_gemm(x, xs, w, ws, dtype=T[kind])
        torch.cuda.synchronize()
        assert st.item() == qamw.QAMW_STATUS_TIMEOUT
        assert (buf[:2048] == -7).all() and (buf[2048 + ntok * d_out:] == -7).all()
        assert torch.equal(got, want)
