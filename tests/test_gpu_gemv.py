"""mx_gemv (bf16 rows times MXFP4 weights) against float64.

On small whole numbers every product and partial sum is an integer multiple
of 1/2 below 2^24, so the fp32 result has to be exact whatever the order.  On
normal values the error of a sum of K fp32 additions in any order is at most
K 2^-23 sum |x w| (one step of 2^-23 an addition leaves room for a matrix core
that truncates), and the bf16 form adds half a step of its own, 2^-8 of the
value.  Every case prints itself before it touches the GPU."""
import sys

import numpy as np
import pytest

from synth import inputs as I
from tests import serving_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X; none is visible")
    import mxfp4_act_quantizer_amd as K
    return K


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def weights(rng, n, k, lo=127, hi=130):
    return (rng.integers(0, 256, (n, k // 2), dtype=np.uint8),
            rng.integers(lo, hi, (n, k // 32), dtype=np.uint8))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 17, 96), (2, 100, 128), (3, 15, 160), (5, 33, 1152), (16, 31, 2240),
          (17, 48, 544), (31, 129, 4096), (33, 64, 96), (47, 5, 8960), (64, 1152, 1152), (64, 77, 32), (1, 4609, 12288),
          (8, 1024, 4640), (1, 7, 65568)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_whole_numbers_are_exact(K, m, n, k, out):
    seed = 100 * m + n + k
    say(f"[gemv whole] m={m} n={n} k={k} out={out} seed={seed}")
    rng = np.random.default_rng(seed)
    top = min(8, max(1, (1 << 24) // (k * 48)))  # |sum| <= K * top * 6 * 4 and halves: below 2^24
    x = rng.integers(-top, top + 1, (m, k)).astype(np.float32)
    qw, sw = weights(rng, n, k)
    want = x.astype(np.float64) @ R.dequant(qw, sw).T
    assert np.abs(want).max() < 2 ** 22
    y = K.mx_gemv(dev(x).bfloat16(), dev(qw), dev(sw), out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    torch.cuda.synchronize()
    assert y.shape == (m, n)
    got = y.float().cpu().numpy()
    if out == "bf16":
        want = torch.from_numpy(want.astype(np.float32)).bfloat16().float().numpy()  # exact float32, one rounding
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("m,n,k", [(1, 640, 1152), (9, 333, 2240), (64, 130, 4608)])
def test_normal_values(K, m, n, k):
    say(f"[gemv normal] m={m} n={n} k={k}")
    rng = np.random.default_rng(7 * m + n)
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).bfloat16()
    qw, sw = R.quantize(rng.standard_normal((n, k)).astype(np.float32) * np.exp(rng.standard_normal((n, 1))))
    w, xd = R.dequant(qw, sw), x.double().numpy()
    want, room = xd @ w.T, k * 2.0 ** -23 * (np.abs(xd) @ np.abs(w).T)
    y32 = K.mx_gemv(x.cuda(), dev(qw), dev(sw))
    y16 = K.mx_gemv(x.cuda(), dev(qw), dev(sw), out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert y32.dtype == torch.float32
    assert (np.abs(y32.cpu().numpy() - want) <= room).all()
    assert torch.equal(y16, y32.bfloat16())  # the same sums, rounded once


def test_extreme_scales_and_nan(K):
    # the smallest and largest scales the quantizer writes, a NaN block, and a zero row
    say("[gemv scales]")
    rng = np.random.default_rng(3)
    n, k = 20, 96
    qw, sw = weights(rng, n, k)
    qw[:6] = 0x11  # value 1/2 each
    sw[0], sw[1], sw[2] = 0, 1, 252
    sw[3] = 127
    sw[3, 1] = 255
    qw[4] = 0
    x = np.ones((2, k), np.float32)
    x[1] = 2.0
    y = K.mx_gemv(dev(x).bfloat16(), dev(qw), dev(sw)).cpu().numpy().astype(np.float64)
    for r, f in ((0, 1.0), (1, 2.0)):
        assert y[r, 0] == f * 96 * 0.5 * 2.0 ** -127
        assert y[r, 1] == f * 96 * 0.5 * 2.0 ** -126
        assert y[r, 2] == f * 96 * 0.5 * 2.0 ** 125 if f * 48 * 2.0 ** 125 < 2.0 ** 128 else np.isinf(y[r, 2])
        assert np.isnan(y[r, 3]) and y[r, 4] == 0.0
    assert np.isfinite(y[:, 5:]).all()  # the NaN stays in its row


def test_rows_do_not_mix(K):
    # an infinity and a NaN in one row of x, and guard values around the output
    say("[gemv rows]")
    rng = np.random.default_rng(4)
    m, n, k = 18, 50, 256
    x = rng.standard_normal((m, k)).astype(np.float32)
    qw, sw = weights(rng, n, k)
    clean = K.mx_gemv(dev(x).bfloat16(), dev(qw), dev(sw))
    x[3, 7], x[17, 200] = np.inf, np.nan
    buf = torch.full((m * n + 64,), 7.5, device="cuda")
    out = buf[32:32 + m * n].view(m, n)
    K.mx_gemv(dev(x).bfloat16(), dev(qw), dev(sw), out=out)
    torch.cuda.synchronize()
    keep = [r for r in range(m) if r not in (3, 17)]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[3]).any() and torch.isnan(out[17]).all()
    assert (buf[:32] == 7.5).all() and (buf[32 + m * n:] == 7.5).all()


def test_views_streams_and_graph(K):
    # buffers at the least alignment, another stream, and a captured call replayed on new inputs
    say("[gemv graph]")
    rng = np.random.default_rng(5)
    m, n, k = 4, 300, 1152
    qw, sw = weights(rng, n, k)
    x = dev(rng.integers(-3, 4, (m, k)).astype(np.float32)).bfloat16()
    odd = torch.empty(sw.size + 3, dtype=torch.uint8, device="cuda")
    swd = odd[3:].view(n, k // 32)
    swd.copy_(dev(sw))
    want = K.mx_gemv(x, dev(qw), dev(sw))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    flat = torch.zeros(m * n + 1, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    got = K.mx_gemv(x, dev(qw), swd, out=flat[1:].view(m, n), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, qd = torch.zeros((m, n), device="cuda"), dev(qw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.mx_gemv(x, qd, swd, out=out)
    for i in range(4):
        x.copy_(dev(rng.integers(-3, 4, (m, k)).astype(np.float32)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, K.mx_gemv(x, qd, swd)), i


def test_feeds_the_adaln_front_end(K):
    """The modulation linear of two samples, then the quantizer it feeds: the
    shift and scale halves of one float32 product go straight into
    kq_adaln_quantize, and the result equals the same call on the float64
    product rounded to float32 wherever the two agree bit for bit."""
    say("[gemv adaln]")
    d, samples, T = 1152, 2, 64
    rng = np.random.default_rng(6)
    cond = rng.integers(-4, 5, (samples, d)).astype(np.float32)
    qw, sw = weights(rng, 2 * d, d, lo=117, hi=120)
    mod = K.mx_gemv(dev(cond).bfloat16(), dev(qw), dev(sw))
    want = cond.astype(np.float64) @ R.dequant(qw, sw).T  # exact in float32 (whole multiples of 2^-11)
    np.testing.assert_array_equal(mod.cpu().numpy(), want)
    h = I.act_dit_lognormal(samples * T, d, 9)[0]
    hd = dev(h.view(np.int16)).view(torch.bfloat16)
    f = dev(I.random_factors(d // 32, 10))
    shift, scale = mod[:, :d].contiguous(), mod[:, d:].contiguous()
    q, s = K.kq_adaln_quantize(hd, shift, scale, T, 1e-6, f)
    w = dev(want.astype(np.float32))
    q2, s2 = K.kq_adaln_quantize(hd, w[:, :d].contiguous(), w[:, d:].contiguous(), T, 1e-6, f)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
