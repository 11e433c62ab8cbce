"""mx_cache_attention against float64 (tests/serving_ref.py states how far off
it may be and why).

Cache slots that no sequence position owns hold hostile bytes: random codes
under NaN scales and the largest scales, so a kernel that lets an unseen
position through, even with weight zero, returns NaN.  Every case prints
itself before it touches the GPU."""
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


class Setup:
    """A batch over a cache whose owned slots hold quantized normal values and
    whose other slots are hostile."""

    def __init__(self, rng, new, lengths, q_heads, heads, dim, size, spare=3):
        need = [-(-max(n, 0) // size) for n in lengths]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(new), max(need + [1])), order[-1], np.int32)  # unused entries: a hostile page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lengths = np.asarray(lengths, np.int32)
        self.rows = int(self.start[-1])
        shape = (self.pages, heads, size)
        self.buf = []
        for _ in "kv":
            codes = rng.integers(0, 256, (*shape, dim // 2), dtype=np.uint8)
            scales = rng.choice(np.array([255, 254, 0], np.uint8), (self.pages, heads, dim // 32, size))
            x = rng.standard_normal((*shape, dim)) * np.exp(0.5 * rng.standard_normal((*shape, 1)))
            c, s = R.quantize(x.astype(np.float32))
            for i, n in enumerate(lengths):
                for j in range(n):
                    pg, of = self.table[i, j // size], j % size
                    codes[pg, :, of], scales[pg, :, :, of] = c[pg, :, of], s[pg, :, of]
            self.buf += [codes, scales]
        q = rng.standard_normal((self.rows, q_heads, dim)).astype(np.float32) * 2.0
        self.q = torch.from_numpy(q).bfloat16()
        self.dim = dim

    def args(self, K):
        return (K.MXCache(*(dev(b) for b in self.buf)), i32(self.table), i32(self.start), i32(self.lengths))

    def want(self, scale=None, window=0, sinks=0):
        return R.attention(self.q.double().numpy(), *self.buf, self.table, self.start, self.lengths,
                           self.dim ** -0.5 if scale is None else scale, window, sinks)

    def check(self, K, scale=None, window=0, sinks=0):
        got = K.mx_cache_attention(self.q.cuda(), *self.args(K), softmax_scale=scale, window=window, sinks=sinks)
        torch.cuda.synchronize()
        compare(got, *self.want(scale, window, sinks))
        return got


def compare(got, want, room):
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want)), (np.isnan(g).sum(), np.isnan(want).sum())
    off = np.where(np.isnan(want), 0.0, np.abs(g - want) - room)
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:5])


# new rows, lengths, query heads, heads, page size
BATCHES = [
    ([1], [1], 1, 1, 16), ([1], [33], 4, 1, 16), ([1, 1, 1], [31, 32, 64], 8, 8, 32), ([2], [2], 6, 2, 16),
    ([1, 1], [257, 15], 10, 2, 48), ([3, 1, 0, 2], [40, 100, 7, 2], 6, 3, 64),  # a few columns
    ([5, 7], [90, 7], 16, 4, 16), ([1], [70], 34, 2, 128),                      # two column tiles a wave
    ([70, 1], [200, 3], 2, 1, 16), ([33], [33], 12, 3, 80), ([130, 64, 1], [131, 90, 500], 4, 2, 1024),  # wide tiles
    ([1], [3001], 2, 1, 16), ([4, 1], [2500, 700], 4, 2, 256)]                  # split over workgroups


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,lengths,q_heads,heads,size", BATCHES)
def test_causal(K, new, lengths, q_heads, heads, size, dim):
    say(f"[attention] new={new} lengths={lengths} heads={q_heads}/{heads} dim={dim} page={size}")
    rng = np.random.default_rng(sum(lengths) + dim)
    Setup(rng, new, lengths, q_heads, heads, dim, size).check(K)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (32, 0), (33, 40), (100, 4), (64, 33), (700, 5),
                                          (1 << 30, 9), (200, 1 << 30)])
def test_window_and_sinks(K, window, sinks, dim):
    say(f"[attention window] window={window} sinks={sinks} dim={dim}")
    rng = np.random.default_rng(window % 1000 + sinks % 1000 + dim)
    for new, lengths, q_heads, heads in (([1, 1, 1], [600, 33, 1], 4, 2), ([90, 3], [601, 3], 4, 2),
                                         ([12], [300], 4, 1)):
        Setup(rng, new, lengths, q_heads, heads, dim, 48).check(K, window=window, sinks=sinks)


@pytest.mark.parametrize("scale", [1e-4, 0.05, 3.0, 40.0])
def test_scales(K, scale):
    # nearly uniform weights, and weights that underflow all but one
    say(f"[attention scale] {scale}")
    rng = np.random.default_rng(11)
    Setup(rng, [1, 40], [900, 300], 4, 2, 128, 32).check(K, scale=scale)


def test_rising_scores(K):
    """Keys whose scores rise (and fall) along the sequence, so that the
    running maximum is raised again and again, and stays behind by less than
    the threshold in between."""
    say("[attention rising]")
    rng = np.random.default_rng(12)
    for sign in (1, -1):
        s = Setup(rng, [1, 20], [1500, 1500], 2, 1, 64, 64)
        for i in range(2):
            for j in range(1500):
                x = np.full((1, 64), 6.0 * sign * (j - 750) / 750, np.float32)
                x += rng.standard_normal(x.shape).astype(np.float32) * 0.1
                pg, of = s.table[i, j // 64], j % 64
                s.buf[0][pg, :, of], s.buf[1][pg, :, :, of] = R.quantize(x)
        s.q = torch.ones_like(s.q)
        s.check(K)


def test_rows_that_see_nothing(K):
    """Positions before 0, lengths of zero, pages out of range, lengths past
    the table, rows of no sequence."""
    say("[attention empty rows]")
    rng = np.random.default_rng(13)
    s = Setup(rng, [4, 1, 3, 40, 2], [2, 0, 100, 90, 112], 4, 2, 64, 16)
    s.table[2, 1:3] = [-1, s.pages]  # positions 16..47 of sequence 2 have no slot
    s.table[3, 0] = 0x7FFFFFFF
    assert s.table.shape[1] == 7
    s.lengths[4] = 112 + 40  # both rows lie past the table's 112 positions
    want, room = s.want()
    assert (want[:2] == 0).all() and (want[4] == 0).all()
    got = s.check(K)
    assert (got[:2] == 0).all() and (got[4] == 0).all()
    s.check(K, window=20, sinks=3)  # sequence 4 then sees its sinks alone
    # rows of no sequence keep what they held
    extra = torch.cat([s.q, s.q[:5]]).cuda()
    out = torch.full_like(extra, 33.0)
    K.mx_cache_attention(extra, *s.args(K), out=out)
    compare(out[:s.rows], want, room)
    assert (out[s.rows:] == 33).all()
    # every page out of range, and a table of no width
    c, table, start, lengths = s.args(K)
    assert (K.mx_cache_attention(s.q.cuda(), c, torch.full_like(table, -1), start, lengths) == 0).all()
    assert (K.mx_cache_attention(s.q.cuda(), c, table[:, :0].contiguous(), start, lengths) == 0).all()


@pytest.mark.parametrize("rows", [1, 3])
def test_extreme_lengths(K, rows):
    """The smallest and largest 32-bit lengths, and lengths just below and
    above zero: negative positions see nothing, positions far past the table
    see all of it."""
    say(f"[attention extreme lengths] rows={rows}")
    rng = np.random.default_rng(23)
    s = Setup(rng, [rows] * 6, [64] * 6, 4, 2, 64, 16)
    s.lengths[:] = [-2 ** 31, -2 ** 31 + 1, -1, 0, 2 ** 31 - 1, 64]
    s.table[:] = s.table[4]  # positions past a length must not matter: every page is one of sequence 4's
    want, _ = s.want()
    assert (want[:4 * rows] == 0).all() and (want[4 * rows:] != 0).any()
    got = s.check(K)
    assert (got[:4 * rows] == 0).all()
    s.check(K, window=30, sinks=2)
    s.check(K, window=1 << 30, sinks=1 << 30)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_stays_where_it_is_seen(K, dim):
    """NaN blocks in keys and values, a NaN and an infinity in q: only rows
    that see them change, and of V only the block's channels."""
    say(f"[attention nan] dim={dim}")
    rng = np.random.default_rng(14)
    for new, lengths, q_heads, heads in (([40, 1], [70, 41], 4, 2), ([6, 1], [70, 41], 2, 1), ([1, 1], [70, 41], 2, 2)):
        s = Setup(rng, new, lengths, q_heads, heads, dim, 16)

        def put(which, seq, j, head, blk):
            pg, of = s.table[seq, j // 16], j % 16
            s.buf[which + 1][pg, head, blk, of] = 255
            s.buf[which][pg, head, of, blk * 16:(blk + 1) * 16] = 0

        put(2, 0, 67, heads - 1, 1)      # a value that only the last rows see
        put(2, 0, 68, 0, dim // 32 - 1)
        put(0, 0, 69, 0, 0)              # the last row's own key
        put(0, 1, 40, heads - 1, 0)
        s.q[0, 0, 3] = float("nan")
        want, _ = s.want()
        assert np.isnan(want).any() and not np.isnan(want).all()
        got = s.check(K)
        s.check(K, window=2)
        s.q[0, 0, 3] = float("inf")
        g = K.mx_cache_attention(s.q.cuda(), *s.args(K))
        assert torch.isnan(g[0, 0]).all() and torch.equal(g[1:].isnan(), got[1:].isnan())


def test_strides_streams_workspace(K):
    """q and out as slices, one workspace for calls in turn, another stream;
    equal bits every time, guard values around the output."""
    say("[attention views]")
    rng = np.random.default_rng(15)
    s = Setup(rng, [1, 1, 2], [2000, 64, 900], 4, 2, 128, 32)
    args = s.args(K)
    want = s.check(K)
    qkv = torch.full((s.rows, 9, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:6] = s.q.cuda()
    out = torch.full((s.rows + 2, 7, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    need = K.mx_cache_attention_workspace(s.rows, 4, *args)
    assert need > 0
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN bits
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        K.mx_cache_attention(qkv[:, 2:6], *args, out=out[1:-1, 3:], workspace=work[:need], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out[1:-1, 3:], want)
        assert (out[:, :3] == 9).all() and (out[0] == 9).all() and (out[-1] == 9).all()
        assert (work[need:] == 0xFF).all()
    with pytest.raises(K.KQError):
        K.mx_cache_attention(s.q.cuda(), *args, workspace=work[:need - 16])
    with pytest.raises(ValueError):
        K.mx_cache_attention(qkv[:, ::2][:, :4], *args)


def test_buffers_belong_to_the_calls_stream(K):
    """What a call allocates comes from the memory of the stream it runs on:
    the workspace is freed when the call returns, and its bytes then go to
    that stream's next work, not to the current stream's."""
    say("[attention buffers of a stream]")
    rng = np.random.default_rng(24)
    s = Setup(rng, [1, 1], [4000, 64], 4, 2, 128, 32)
    args, q = s.args(K), s.q.cuda()
    want = s.check(K)
    x = torch.ones((1, 128), dtype=torch.bfloat16, device="cuda")
    qw, sw = (torch.zeros((64, n), dtype=torch.uint8, device="cuda") for n in (64, 4))
    need = K.mx_cache_attention_workspace(s.rows, 4, *args)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = K.mx_cache_attention(q, *args, stream=side)
    k, v = K.mx_cache_read(*args, rows=s.rows, stream=side)
    y = K.mx_gemv(x, qw, sw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (y == 0).all()
    segments = [g for g in torch.cuda.memory_snapshot() if g["stream"] == side.cuda_stream]
    for t in (out, k, v, y):
        assert any(0 <= t.data_ptr() - g["address"] < g["total_size"] for g in segments)
    assert max(b["size"] for g in segments for b in g["blocks"] if b["state"] != "active_allocated") >= need


def test_usual_calls_and_the_rest_agree(K):
    """The compiled host side of the usual call and the Python side that takes
    every other: the same bits, the same errors."""
    say("[attention host sides]")
    rng = np.random.default_rng(27)
    s = Setup(rng, [2, 1], [700, 33], 4, 2, 64, 16)
    args, q = s.args(K), s.q.cuda()
    cache = args[0]
    here = torch.cuda.current_stream()
    want = K.mx_cache_attention(q, *args, softmax_scale=0.2, window=100, sinks=3, stream=here)
    assert torch.equal(K.mx_cache_attention(q, *args, softmax_scale=0.2, window=100, sinks=3), want)
    out = torch.zeros_like(q)
    assert K.mx_cache_attention(q, *args, softmax_scale=0.2, window=100, sinks=3, out=out) is out
    assert torch.equal(out, want)
    bits = K.mx_cache_attention(q.view(torch.int16), *args, softmax_scale=np.float64(0.2), window=100, sinks=3)
    assert torch.equal(bits, want)
    plain = K.mx_cache_attention(q, *args)
    assert torch.equal(plain, K.mx_cache_attention(q, *args, stream=here))
    for a, b in zip(K.mx_cache_read(*args, rows=s.rows), K.mx_cache_read(*args, rows=s.rows, stream=here)):
        assert a.dtype == torch.bfloat16 and torch.equal(a, b)
    copies = [K.MXCache(*(t.clone() for t in cache)) for _ in range(2)]
    kv = torch.from_numpy(rng.standard_normal((s.rows, 2, 64)).astype(np.float32)).bfloat16().cuda()
    f = dev(I.random_factors(1, 28))
    for c, stream in zip(copies, (None, here)):
        assert K.mx_cache_write(kv, kv, c, *args[1:], factors=f, stream=stream) is None
    for a, b in zip(*copies):
        assert torch.equal(a, b)
    x = torch.randn((3, 128), device="cuda").bfloat16()
    w = [torch.randint(100, 130, shape, dtype=torch.uint8, device="cuda") for shape in ((40, 64), (40, 4))]
    for dtype in (torch.float32, torch.bfloat16):
        y = K.mx_gemv(x, *w, out_dtype=dtype)
        assert y.dtype == dtype and torch.equal(y, K.mx_gemv(x, *w, out_dtype=dtype, stream=here))
        z = torch.zeros_like(y)
        assert K.mx_gemv(x, *w, out=z) is z and torch.equal(y, z)
    assert K.mx_gemv(x, *w).dtype == torch.float32
    for stream in (None, here):
        for bad in (dict(softmax_scale=0.0), dict(window=-1), dict(out=q[:2]), dict(out=q), dict(window=1 << 64),
                    dict(window=7, sinks=-(1 << 70))):
            with pytest.raises((K.KQError, ValueError)):
                K.mx_cache_attention(q, *args, stream=stream, **bad)
        for call in (lambda: K.mx_gemv(x, w[0][:20], w[1], stream=stream),
                     lambda: K.mx_gemv(x, *w, out_dtype=torch.float16, stream=stream),
                     lambda: K.mx_gemv(x, *w, out=y, out_dtype=torch.float32, stream=stream),
                     lambda: K.mx_cache_write(kv, kv[:1], cache, *args[1:], stream=stream),
                     lambda: K.mx_cache_read(cache, args[1], args[3], args[2], rows=2, stream=stream)):
            with pytest.raises(ValueError):
                call()
        for call in (lambda: K.mx_gemv(x.cpu(), *w, stream=stream), lambda: K.mx_gemv(x, w[0].int(), w[1], stream=stream),
                     lambda: K.mx_gemv(x.float(), *w, stream=stream),
                     lambda: K.mx_cache_write(kv.float(), kv, cache, *args[1:], stream=stream),
                     lambda: K.mx_cache_read(cache, args[1].long(), *args[2:], rows=2, stream=stream)):
            with pytest.raises(TypeError):
                call()


def test_graph_decodes_a_growing_sequence(K):
    """One captured step (write, then attention) replayed while the lengths
    grow through pages and tiles; every replay equals the eager call."""
    say("[attention graph]")
    rng = np.random.default_rng(16)
    heads, q_heads, dim, size, width = 2, 8, 64, 16, 40
    cache = K.mx_cache_new(2 * width, size, heads, dim)
    table = i32(rng.permutation(2 * width).reshape(2, width))
    start, lengths = i32([0, 1, 2]), i32([0, 290])
    qkv = torch.zeros((2, q_heads + 2 * heads, dim), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((2, q_heads, dim), dtype=torch.bfloat16, device="cuda")
    work = torch.empty(max(1, K.mx_cache_attention_workspace(2, q_heads, cache, table, start, lengths)),
                       dtype=torch.uint8, device="cuda")

    def step():
        K.mx_cache_write(qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:], cache, table, start, lengths)
        K.mx_cache_attention(qkv[:, :q_heads], cache, table, start, lengths, out=out, workspace=work)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(40):
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)))
        lengths += 1
        g.replay()
        torch.cuda.synchronize()
        if i % 3 == 0 or i > 36:
            eager = K.mx_cache_attention(qkv[:, :q_heads].contiguous(), cache, table, start, lengths)
            assert torch.equal(out, eager), i
    want, room = R.attention(qkv[:, :q_heads].double().cpu().numpy(), *(b.cpu().numpy() for b in cache),
                             table.cpu().numpy(), [0, 1, 2], lengths.cpu().numpy(), dim ** -0.5)
    compare(out, want, room)


@pytest.mark.parametrize("dim,q_heads,heads", [(64, 2, 2), (128, 4, 1), (256, 3, 1), (128, 24, 1)])
def test_shares_end_anywhere(K, dim, q_heads, heads):
    """Sequences of very different lengths, short and empty ones among long
    ones: the equal shares of the work then begin and end inside them."""
    say(f"[attention shares] dim={dim} heads={q_heads}/{heads}")
    rng = np.random.default_rng(21)
    new = [1, 1, 1, 2, 0, 1, 3, 1, 1, 1, 2, 1]
    lengths = [3000, 5, 0, 1700, 40, 2200, 64, 3100, 1, 1601, 2, 1537]
    s = Setup(rng, new, lengths, q_heads, heads, dim, 128)
    s.check(K)
    s.check(K, window=1800, sinks=70)
    s.check(K, window=300, sinks=5)


@pytest.mark.parametrize("new,q_heads", [(1, 4), (90, 2)])
def test_row_starts_that_decrease(K, new, q_heads):
    """A row_start that goes back and forth: its rows may count as anybody's,
    but nothing outside the output's rows is written, and the call after it is
    right."""
    say(f"[attention decreasing starts] new={new}")
    rng = np.random.default_rng(25)
    s = Setup(rng, [new] * 9, [2000] * 9, q_heads, 1, 64, 64)
    c, table, start, lengths = s.args(K)
    n = s.rows
    bad = [0, n, 0, n, n // 2, n, -5, n + 7, 0, n]
    out = torch.full((n + 2, q_heads, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    K.mx_cache_attention(s.q.cuda(), c, table, i32(bad), lengths, out=out[1:-1])
    torch.cuda.synchronize()
    assert (out[0] == 9).all() and (out[-1] == 9).all()
    s.check(K)


@pytest.mark.parametrize("dim,lengths", [(64, [3000, 90, 1700, 400]), (128, [5000]), (256, [2600, 300])])
def test_chunks_share_the_work(K, dim, lengths):
    """Chunks whose column tiles are cut between workgroups."""
    say(f"[attention chunk shares] dim={dim} lengths={lengths}")
    rng = np.random.default_rng(26)
    s = Setup(rng, [85, 70, 131, 129][:len(lengths)], lengths, 3, 1, dim, 112)
    s.check(K)
    s.check(K, window=1500, sinks=40)


def test_more_sequences_than_a_line(K):
    # long sequences, and one more of them than the shares are made for
    say("[attention 257 sequences]")
    rng = np.random.default_rng(22)
    new = [1] * 257
    lengths = [1 + (37 * i) % 90 for i in range(256)] + [2100]
    Setup(rng, new, lengths, 2, 1, 64, 64).check(K)
    Setup(rng, new[1:], lengths[1:], 2, 1, 64, 64).check(K)


def test_many_sequences(K):
    say("[attention many]")
    rng = np.random.default_rng(17)
    seqs = 700  # past the count that is split, and past two rounds of the search
    new = [int(n) for n in rng.integers(0, 3, seqs)]
    lengths = [n + int(x) for n, x in zip(new, rng.integers(0, 30, seqs))]
    Setup(rng, new, lengths, 2, 1, 64, 16).check(K)


def test_offsets_past_32_bits(K):
    say("[attention large]")
    heads, dim, size, pages = 8, 256, 1024, 4200
    cache = K.mx_cache_new(pages, size, heads, dim)
    assert cache.kq.numel() > 1 << 32
    rng = np.random.default_rng(18)
    x = [torch.from_numpy(rng.standard_normal((1500, heads, dim)).astype(np.float32)).bfloat16().cuda() for _ in "kv"]
    q = torch.from_numpy(rng.standard_normal((3, 16, dim)).astype(np.float32)).bfloat16()
    table, lengths = np.array([[pages - 1, pages - 3]], np.int32), np.array([1500], np.int32)
    K.mx_cache_write(*x, cache, i32(table), i32([0, 1500]), i32(lengths))
    got = K.mx_cache_attention(q.cuda(), cache, i32(table), i32([0, 3]), i32(lengths))
    small = [b[[pages - 1, pages - 3]].cpu().numpy() for b in cache]
    compare(got, *R.attention(q.double().numpy(), *small, np.array([[0, 1]]), [0, 3], lengths, dim ** -0.5))


def test_a_whole_step(K):
    """The operators as they are used together: a fused projection by mx_gemv,
    keys rotated as they are cached and queries by the transposed inverse,
    attention, and the output projection; against the same step in float64
    from the cached values that mx_cache_read gives back."""
    say("[attention step]")
    rng = np.random.default_rng(19)
    width, heads, q_heads, dim, size, seqs = 256, 2, 4, 64, 16, 3
    wqkv = R.quantize(rng.standard_normal(((q_heads + 2 * heads) * dim, width)).astype(np.float32) / 16)
    wout = R.quantize(rng.standard_normal((width, q_heads * dim)).astype(np.float32) / 16)
    f = I.random_factors(heads * dim // 32, 20)
    turn = np.swapaxes(K.kq_factor_inverse(f), 2, 3)
    # one set for each block of a key; the query heads that share a key head share its sets
    turn = np.repeat(turn.reshape(heads, 1, dim // 32, 5, 2, 2), q_heads // heads, 1).reshape(-1, 5, 2, 2)
    fd, turnd = dev(f), dev(turn)
    cache = K.mx_cache_new(3 * 5, size, heads, dim)
    table, start = i32(rng.permutation(15).reshape(seqs, 5)), i32(np.arange(seqs + 1))
    lengths = i32([0, 5, 40])
    for step in range(30):
        lengths += 1
        x = torch.from_numpy(rng.standard_normal((seqs, width)).astype(np.float32)).bfloat16().cuda()
        qkv = K.mx_gemv(x, dev(wqkv[0]), dev(wqkv[1]), out_dtype=torch.bfloat16).view(seqs, -1, dim)
        q, k, v = qkv.split([q_heads, heads, heads], 1)
        K.mx_cache_write(k, v, cache, table, start, lengths, factors=fd)
        qt = K.kq_transform_f32(q.reshape(seqs, -1).contiguous(), turnd).bfloat16().view(seqs, q_heads, dim)
        o = K.mx_cache_attention(qt, cache, table, start, lengths)
        y = K.mx_gemv(o.view(seqs, -1), dev(wout[0]), dev(wout[1]))
    want, room = R.attention(qt.double().cpu().numpy(), *(b.cpu().numpy() for b in cache), table.cpu().numpy(),
                             np.arange(seqs + 1), lengths.cpu().numpy(), dim ** -0.5)
    compare(o, want, room)
    w = R.dequant(*wout)
    on = o.double().cpu().numpy().reshape(seqs, -1)
    off = np.abs(y.double().cpu().numpy() - on @ w.T)
    assert (off <= w.shape[1] * 2.0 ** -23 * (np.abs(on) @ np.abs(w).T)).all()
    # the rotation leaves the scores: q . k of the last token, from the unrotated values and from the rotated ones
    kr, _ = K.mx_cache_read(cache, table, start, lengths, rows=seqs)
    kf = K.kq_transform_f32(k.reshape(seqs, -1).contiguous(), fd).view(seqs, heads, dim)
    plain = (q.double().view(seqs, heads, -1, dim) * k.double().view(seqs, heads, 1, dim)).sum(-1)
    turned = (qt.double().view(seqs, heads, -1, dim) * kf.double().view(seqs, heads, 1, dim)).sum(-1)
    size_of = (qt.double().abs().view(seqs, heads, -1, dim) * kf.double().abs().view(seqs, heads, 1, dim)).sum(-1)
    # the queries' rounding to bf16 (2^-8 of each product) and fp32 transforms
    assert ((plain - turned).abs() <= (2.0 ** -8 + 2.0 ** -16) * size_of).all()
    # a quantized block is within half its largest step of what was written: 2 units of 2^(s - 127), 4 at the top
    blocks = (kr.double() - kf.double()).abs().view(-1, 32).amax(1)
    top = kf.double().abs().view(-1, 32).amax(1)
    assert (blocks <= top * (0.25 + 2.0 ** -16)).all()
