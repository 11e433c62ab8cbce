"""The paged MXFP4 cache: mx_cache_write and mx_cache_read.

Codes and scales are compared bit for bit with the oracle's quantizer (plain
rows), with kq_quantize_ex(KQ_VARIANT_BUTTERFLY) at a few thousand blocks
(rotated keys) and with the transform in double at some fifty thousand; reads with
the values that the codes stand for, exactly.  Untouched slots and rows must
keep their bytes.  Every case prints itself before it touches the GPU."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


def batch(rng, new, lengths, size, spare=2):
    """Page table (distinct pages in random order), row_start, lengths, pages."""
    need = [-(-n // size) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(new), max(need + [1])), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), np.asarray(lengths, np.int32), pages


def garbage(rng, pages, heads, size, dim):
    a = [rng.integers(0, 256, s, dtype=np.uint8) for s in 2 * [(pages, heads, size, dim // 2),
                                                              (pages, heads, dim // 32, size)]]
    return a  # kq, ks, vq, vs


def place(buf, page, off, codes, scales):
    buf[0][page, :, off], buf[1][page, :, :, off] = codes, scales


def rows_bf16(rng, rows, heads, dim):
    """bf16 values with outliers, zeros, subnormals; float32 copy beside them."""
    x = rng.standard_normal((rows, heads, dim)).astype(np.float32)
    x[:, :, ::37] *= 40.0
    x[rng.random(x.shape) < 0.01] = -0.0
    if rows > 1:
        x[1] *= 2.0 ** -126
    if rows > 2:
        x[2, 0, :32] = 0.0
    t = torch.from_numpy(x).bfloat16()
    return t, t.float().numpy()


CASES = [  # new rows, lengths, heads, dim, page size
    ([1], [1], 1, 32, 16), ([1, 1, 1], [16, 17, 500], 8, 128, 16), ([5, 0, 40, 1], [5, 9, 100, 64], 2, 64, 48),
    ([130], [130], 5, 32, 16), ([33, 70], [1000, 70], 3, 96, 64), ([7] * 70, list(range(7, 77)), 1, 256, 16),
    ([300, 1, 2], [1300, 1, 2050], 8, 128, 1024), ([9, 3], [10, 3], 4, 160, 80), ([20], [21], 17, 224, 32)]


@pytest.mark.parametrize("new,lengths,heads,dim,size", CASES)
def test_write_then_read(K, new, lengths, heads, dim, size):
    rng = np.random.default_rng(sum(new) + dim)
    say(f"[cache] new={new[:5]} lengths={lengths[:5]} heads={heads} dim={dim} page={size}")
    table, start, length, pages = batch(rng, new, lengths, size)
    rows = int(start[-1])
    kt, kf = rows_bf16(rng, rows, heads, dim)
    vt, vf = rows_bf16(rng, rows, heads, dim)
    want = garbage(rng, pages, heads, size, dim)
    cache = K.MXCache(*(dev(a) for a in want))
    args = (i32(table), i32(start), i32(length))
    K.mx_cache_write(kt.cuda(), vt.cuda(), cache, *args)
    (kc, kscale), (vc, vscale) = R.quantize(kf), R.quantize(vf)
    for r, at in enumerate(R.slots(table, start, length, rows, pages, size)):
        assert at is not None
        place(want[:2], *at, kc[r], kscale[r])
        place(want[2:], *at, vc[r], vscale[r])
    for name, got, w in zip(cache._fields, cache, want):
        np.testing.assert_array_equal(got.cpu().numpy(), w, err_msg=name)
    kr, vr = K.mx_cache_read(cache, *args, rows=rows)
    for got, c, s in ((kr, kc, kscale), (vr, vc, vscale)):
        np.testing.assert_array_equal(got.float().cpu().numpy().astype(np.float64), R.dequant(c, s))


@pytest.mark.parametrize("heads,dim,shared", [(8, 128, False), (3, 96, True), (1, 32, False), (2, 256, True)])
def test_rotated_keys_are_the_quantizers_codes(K, heads, dim, shared):
    rng = np.random.default_rng(heads * dim)
    new, size = [37, 1, 90], 32
    say(f"[cache rotated] heads={heads} dim={dim} shared={shared}")
    table, start, length, pages = batch(rng, new, [50, 1, 90], size)
    rows = int(start[-1])
    kt, _ = rows_bf16(rng, rows, heads, dim)
    vt, vf = rows_bf16(rng, rows, heads, dim)
    f = dev(I.random_factors(1 if shared else heads * dim // 32, 5))
    cache = K.mx_cache_new(pages, size, heads, dim)
    K.mx_cache_write(kt.cuda(), vt.cuda(), cache, i32(table), i32(start), i32(length), factors=f)
    q, s = K.kq_quantize_ex(kt.cuda().view(rows, heads * dim), f, None, None, K.KQ_VARIANT_BUTTERFLY)
    torch.cuda.synchronize()
    q, s = q.cpu().numpy().reshape(rows, heads, -1), s.cpu().numpy().reshape(rows, heads, -1)
    vc, vscale = R.quantize(vf)
    got = [a.cpu().numpy() for a in cache]
    for r, (page, off) in enumerate(R.slots(table, start, length, rows, pages, size)):
        np.testing.assert_array_equal(got[0][page, :, off], q[r])
        np.testing.assert_array_equal(got[1][page, :, :, off], s[r])
        np.testing.assert_array_equal(got[2][page, :, off], vc[r])
        np.testing.assert_array_equal(got[3][page, :, :, off], vscale[r])


def nearest(y):
    """MXFP4 codes and scale bytes of double blocks [..., 32]: thresholds
    between the grid's values, a tie to the even code."""
    amax = np.abs(y).max(-1, keepdims=True)
    e = np.maximum(np.where(amax > 0, np.frexp(amax)[1] - 1, -200) - 2, -127)
    v = np.abs(y) / np.ldexp(1.0, e)
    code = sum((v > t).astype(np.uint8) for t in (0.25, 1.25, 2.5, 5.0))
    code += sum((v >= t).astype(np.uint8) for t in (0.75, 1.75, 3.5))
    code |= (y < 0).astype(np.uint8) << 3
    return code[..., 0::2] | code[..., 1::2] << 4, (e[..., 0] + 127).astype(np.uint8)


@pytest.mark.parametrize("spread", [0, 60])
def test_rotated_keys_are_the_nearest_codes(K, spread):
    """The transform in double and its nearest codes, 1.6 million of them, so
    that some lie at a rounding boundary of fp32's; with `spread`, rows of very
    small and very large values and zero rows."""
    say(f"[cache rotated, nearest] spread={spread}")
    rng = np.random.default_rng(31 + spread)
    rows, heads, dim, size = 1600, 8, 128, 64
    x = rng.standard_normal((rows, heads * dim)).astype(np.float32)
    if spread:
        x *= np.ldexp(np.float32(1), rng.integers(-2 * spread, spread, (rows, 1))).astype(np.float32)
        x[::97] = 0
    kt = torch.from_numpy(x).bfloat16()
    f = I.random_factors(heads * dim // 32, 6)
    cache = K.mx_cache_new(rows // size, size, heads, dim)
    k = kt.cuda().view(rows, heads, dim)
    K.mx_cache_write(k, k, cache, i32([range(rows // size)]), i32([0, rows]), i32([rows]), factors=dev(f))
    y = kt.double().numpy().reshape(rows, -1, 2, 2, 2, 2, 2)
    for axis in range(5):
        a = f.reshape(-1, 5, 2, 2)[:, axis].astype(np.float64)
        u = np.moveaxis(y, 2 + axis, -1)
        u = np.stack([u[..., 0] * a[:, 0, i][:, None, None, None, None] +
                      u[..., 1] * a[:, 1, i][:, None, None, None, None] for i in (0, 1)], -1)
        y = np.moveaxis(u, -1, 2 + axis)
    codes, scales = nearest(y.reshape(rows, heads, dim // 32, 32))
    got = [b.cpu().numpy() for b in cache[:2]]
    at = np.moveaxis(got[0], 1, 2).reshape(rows, heads, dim // 2)
    np.testing.assert_array_equal(np.transpose(got[1], (0, 3, 1, 2)).reshape(scales.shape), scales)
    np.testing.assert_array_equal(at, codes.reshape(at.shape))


def test_nan_and_infinity_blocks(K):
    say("[cache nan]")
    k = torch.ones((2, 2, 64)).bfloat16()
    k[0, 0, 3], k[1, 1, 40] = float("nan"), float("-inf")
    cache = K.mx_cache_new(1, 16, 2, 64)
    args = (i32([[0]]), i32([0, 2]), i32([2]))
    K.mx_cache_write(k.cuda(), torch.ones_like(k).cuda(), cache, *args)
    kr, vr = K.mx_cache_read(cache, *args, rows=2)
    want = torch.ones((2, 2, 64))
    want[0, 0, :32] = float("nan")
    want[1, 1, 32:] = float("nan")
    np.testing.assert_array_equal(kr.float().cpu().numpy(), want.numpy())
    assert (vr == 1).all()
    assert cache.ks[0, 0, 0, 0] == 255 and (cache.kq[0, 0, 0, :16] == 0).all()


def test_rows_without_a_slot(K):
    """Page numbers out of range, lengths too short or too long for the table,
    rows before the first and behind the last sequence, sequences out of
    order: dropped by the write, left as they were by the read."""
    say("[cache slots]")
    rng = np.random.default_rng(1)
    heads, dim, size, pages = 2, 64, 16, 6
    table = np.array([[0, -1, 7], [1, 2, 3], [4, 5, 0x7FFFFFFF], [5, 5, 5]], np.int32)
    start = np.array([2, 42, 47, 53, 50], np.int32)  # sequence 3 runs backwards
    lengths = np.array([40, 3, 50, 9], np.int32)  # 1: its first rows are positions -2, -1; 2: past the table
    rows = 60
    kt, kf = rows_bf16(rng, rows, heads, dim)
    vt, vf = rows_bf16(rng, rows, heads, dim)
    want = garbage(rng, pages, heads, size, dim)
    cache = K.MXCache(*(dev(a) for a in want))
    args = (i32(table), i32(start), i32(lengths))
    where = R.slots(table, start, lengths, rows, pages, size)
    assert sum(w is None for w in where) > 30 and sum(w is not None for w in where) > 15
    K.mx_cache_write(kt.cuda(), vt.cuda(), cache, *args)
    (kc, kscale), (vc, vscale) = R.quantize(kf), R.quantize(vf)
    for r, at in enumerate(where):
        if at:
            place(want[:2], *at, kc[r], kscale[r])
            place(want[2:], *at, vc[r], vscale[r])
    for name, got, w in zip(cache._fields, cache, want):
        np.testing.assert_array_equal(got.cpu().numpy(), w, err_msg=name)
    k0 = torch.full((rows, heads, dim), 77.0, dtype=torch.bfloat16, device="cuda")
    v0 = k0.clone()
    K.mx_cache_read(cache, *args, k=k0, v=v0)
    for r, at in enumerate(where):
        for got, c, s in ((k0, kc, kscale), (v0, vc, vscale)):
            w = R.dequant(c[r], s[r]) if at else np.full((heads, dim), 77.0)
            np.testing.assert_array_equal(got[r].float().cpu().numpy(), w)


def test_extreme_lengths(K):
    # positions at the ends of 32 bits have no slot: nothing is written, nothing read
    say("[cache extreme lengths]")
    rng = np.random.default_rng(6)
    want = garbage(rng, 4, 2, 16, 64)
    cache = K.MXCache(*(dev(a) for a in want))
    kt, _ = rows_bf16(rng, 8, 2, 64)
    args = (i32([[0, 1]] * 4), i32([0, 2, 4, 6, 8]), i32([-2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1, -1]))
    K.mx_cache_write(kt.cuda(), kt.cuda(), cache, *args)
    for got, w in zip(cache, want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    k = torch.full((8, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    K.mx_cache_read(cache, *args, k=k, v=k.clone())
    assert (k == 3).all()


def test_many_sequences(K):
    # more sequences than one and two rounds of the search cover, empty ones among them
    say("[cache many]")
    rng = np.random.default_rng(2)
    seqs, size = 4500, 16
    new = rng.integers(0, 3, seqs)
    lengths = new + rng.integers(0, 20, seqs)
    table, start, length, pages = batch(rng, list(new), list(lengths), size)
    rows = int(start[-1])
    kt, kf = rows_bf16(rng, rows, 1, 32)
    cache = K.mx_cache_new(pages, size, 1, 32)
    args = (i32(table), i32(start), i32(length))
    K.mx_cache_write(kt.cuda(), kt.cuda(), cache, *args)
    kr, vr = K.mx_cache_read(cache, *args, rows=rows)
    want = R.dequant(*R.quantize(kf))
    np.testing.assert_array_equal(kr.float().cpu().numpy(), want)
    np.testing.assert_array_equal(vr.float().cpu().numpy(), want)


def test_slices_whole_sequences_and_graph(K):
    """Keys and values as slices of one projection's output; a chunk at a time,
    then the whole sequences read with their own row_start; the write captured
    and replayed on new rows and moved lengths."""
    say("[cache graph]")
    rng = np.random.default_rng(3)
    heads, dim, size, width = 4, 64, 32, 4
    qkv = torch.zeros((2, 2 + 2 * heads, dim), dtype=torch.bfloat16, device="cuda")  # [rows, q | k | v]
    k, v = qkv[:, 2:2 + heads], qkv[:, 2 + heads:]
    cache = K.mx_cache_new(2 * width, size, heads, dim)
    table, start = i32(rng.permutation(2 * width).reshape(2, width)), i32([0, 1, 2])
    lengths = i32([0, 0])
    K.mx_cache_write(k, v, cache, table, start, lengths)  # lengths 0: no position, nothing written
    assert all((a == 0).all() for a in cache)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.mx_cache_write(k, v, cache, table, start, lengths)
    seen = []
    for i in range(70):
        seen.append(torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)).bfloat16())
        qkv.copy_(seen[-1])
        lengths += i32([1, 1 if i >= 30 else 0])
        g.replay()
        torch.cuda.synchronize()
    kr, vr = K.mx_cache_read(cache, table, i32([0, 70, 110]), lengths, rows=110)
    torch.cuda.synchronize()
    rows = torch.cat([torch.stack([s[0] for s in seen]), torch.stack([s[1] for s in seen[30:]])]).float().numpy()
    # before step 30 sequence 1 has length 0: its row has position -1 and is dropped
    np.testing.assert_array_equal(kr.float().cpu().numpy(), R.dequant(*R.quantize(rows[:, 2:2 + heads])))
    np.testing.assert_array_equal(vr.float().cpu().numpy(), R.dequant(*R.quantize(rows[:, 2 + heads:])))


def test_offsets_past_32_bits(K):
    # a cache whose codes take more than 4 GiB: the last pages are still the last pages
    say("[cache large]")
    heads, dim, size = 8, 256, 1024
    pages = 4200  # 4200 pages x 1 MiB of key codes
    cache = K.mx_cache_new(pages, size, heads, dim)
    assert cache.kq.numel() > 1 << 32
    rng = np.random.default_rng(4)
    kt, kf = rows_bf16(rng, 4, heads, dim)
    table, start, lengths = i32([[pages - 1], [0]]), i32([0, 2, 4]), i32([size, 2])
    K.mx_cache_write(kt.cuda(), kt.cuda(), cache, table, start, lengths)
    c, s = R.quantize(kf)
    np.testing.assert_array_equal(cache.kq[pages - 1, :, size - 2:].cpu().numpy().transpose(1, 0, 2), c[:2])
    np.testing.assert_array_equal(cache.vs[pages - 1, :, :, size - 2:].cpu().numpy().transpose(2, 0, 1), s[:2])
    np.testing.assert_array_equal(cache.kq[0, :, :2].cpu().numpy().transpose(1, 0, 2), c[2:])
    kr, _ = K.mx_cache_read(cache, table, start, lengths, rows=4)
    np.testing.assert_array_equal(kr.float().cpu().numpy(), R.dequant(c, s))
