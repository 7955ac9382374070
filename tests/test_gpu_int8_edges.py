"""The 8-bit (W8A8) operators where they are easily wrong: waits that give up, buffers that the
call ahead has just written, the ends of the range, first calls from several host threads."""
import numpy as np
import pytest
import torch

from tests import int8_ref as ref
from tests.test_gpu_int8 import DEV, T, status, values
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
