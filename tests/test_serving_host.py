"""Argument checks of the few-row product and of the paged cache: every one
returns before any HIP call, so they run without a GPU."""
import ctypes

import pytest

import mxfp4_act_quantizer_amd as K


class CacheArg(ctypes.Structure):  # mx_cache in kroquant.h
    _fields_ = [(f, ctypes.c_void_p) for f in ("kq", "ks", "vq", "vs")] + [
        (f, ctypes.c_int64) for f in ("pages", "page_size", "heads", "dim")]


class BatchArg(ctypes.Structure):  # mx_batch
    _fields_ = [(f, ctypes.c_void_p) for f in ("page_table", "row_start", "lengths")] + [
        (f, ctypes.c_int64) for f in ("seqs", "width", "rows")]


FAKE = 1 << 40  # never dereferenced: every call below fails validation first
GIB = 1 << 30


def raw(name, *args):
    return getattr(K.lib(), name)(*args)


def cache(**kw):
    c = dict(kq=FAKE, ks=FAKE + GIB, vq=FAKE + 2 * GIB, vs=FAKE + 3 * GIB, pages=10, page_size=16, heads=2, dim=64)
    c.update(kw)
    return ctypes.byref(CacheArg(**c))


def batch(**kw):
    b = dict(page_table=FAKE + 4 * GIB, row_start=FAKE + 5 * GIB, lengths=FAKE + 6 * GIB, seqs=3, width=4, rows=7)
    b.update(kw)
    return ctypes.byref(BatchArg(**b))


def test_gemv_refusals():
    x, qw, sw, o = (FAKE + i * GIB for i in range(4))

    def call(x=x, M=4, qw=qw, sw=sw, N=64, K_=128, out=o, bf=0):
        return raw("mx_gemv", x, M, qw, sw, N, K_, out, bf, None)

    assert call(M=-1) == call(N=-1) == call(K_=0) == call(bf=2) == K.KQ_ERR_ARG
    assert call(x=None) == call(qw=None) == call(sw=None) == call(out=None) == K.KQ_ERR_ARG
    assert call(K_=48) == call(M=K.KQ_GEMV_MAX_ROWS + 1) == call(N=(1 << 21) + 1) == K.KQ_ERR_SHAPE
    assert call(K_=(1 << 20) + 32) == K.KQ_ERR_SHAPE
    assert call(x=x + 8) == call(qw=qw + 8) == call(out=o + 2) == call(out=o + 1, bf=1) == K.KQ_ERR_ALIGN
    assert call(out=x + 64) == call(out=qw + 64) == call(out=sw + 4) == K.KQ_ERR_OVERLAP
    assert call(M=0, x=None, out=None) == call(N=0, qw=None) == K.KQ_OK


@pytest.mark.parametrize("name", ["write", "read"])
def test_cache_refusals(name):
    k, v = FAKE + 7 * GIB, FAKE + 8 * GIB

    def call(c=None, b=None, k=k, v=v):
        c, b = c or cache(), b or batch()
        if name == "write":
            return raw("mx_cache_write", k, 128, v, 128, None, 1, c, b, None)
        return raw("mx_cache_read", c, b, k, v, None)

    for f in ("pages", "page_size", "heads", "dim"):
        assert call(cache(**{f: 0})) == call(cache(**{f: -1})) == K.KQ_ERR_ARG, f
    for f in ("kq", "ks", "vq", "vs"):
        assert call(cache(**{f: None})) == K.KQ_ERR_ARG, f
        assert call(cache(**{f: FAKE + 40 * GIB + 8})) == K.KQ_ERR_ALIGN, f
    assert call(cache(dim=48)) == call(cache(dim=288)) == call(cache(page_size=24)) == K.KQ_ERR_SHAPE
    assert call(cache(page_size=1040)) == call(cache(heads=1025)) == call(cache(pages=1 << 31)) == K.KQ_ERR_SHAPE
    for f in ("seqs", "width", "rows"):
        assert call(b=batch(**{f: -1})) == K.KQ_ERR_ARG, f
    for f in ("page_table", "row_start", "lengths"):
        assert call(b=batch(**{f: None})) == K.KQ_ERR_ARG, f
        assert call(b=batch(**{f: FAKE + 40 * GIB + 2})) == K.KQ_ERR_ALIGN, f
    assert call(b=batch(rows=(1 << 28) + 1)) == call(b=batch(seqs=(1 << 20) + 1)) == K.KQ_ERR_SHAPE
    assert call(b=batch(width=(1 << 26) + 1)) == K.KQ_ERR_SHAPE
    assert call(k=None) == call(v=None) == K.KQ_ERR_ARG
    assert call(k=k + 8) == call(v=v + 8) == K.KQ_ERR_ALIGN
    # outputs inside inputs or each other
    assert call(k=FAKE + 64) == call(v=FAKE + 3 * GIB) == K.KQ_ERR_OVERLAP
    assert call(cache(ks=FAKE + 7 * GIB)) == K.KQ_ERR_OVERLAP
    if name == "write":
        assert call(cache(vq=FAKE + 128)) == call(b=batch(lengths=FAKE + 16)) == K.KQ_ERR_OVERLAP
    else:
        assert call(v=k + 128) == call(b=batch(lengths=v + 16)) == K.KQ_ERR_OVERLAP
    for empty in (batch(rows=0), batch(seqs=0, page_table=None, row_start=None, lengths=None)):
        assert call(b=empty, k=None, v=None) == K.KQ_OK


def test_cache_write_strides_and_factors():
    k, v, f = FAKE + 7 * GIB, FAKE + 8 * GIB, FAKE + 9 * GIB

    def call(ks=128, vs=128, factors=None, nT=1, c=None):
        return raw("mx_cache_write", k, ks, v, vs, factors, nT, c or cache(), batch(), None)

    assert call(ks=120) == call(vs=64) == call(ks=(1 << 31) + 8) == K.KQ_ERR_SHAPE
    assert call(ks=132) == call(vs=129) == K.KQ_ERR_ALIGN
    assert call(factors=f, nT=2) == call(factors=f, nT=0) == K.KQ_ERR_SHAPE
    assert call(factors=f + 2, nT=4) == K.KQ_ERR_ALIGN
    assert call(factors=FAKE + 8, nT=4) == K.KQ_ERR_OVERLAP
    # the last row of a strided view counts: 6 rows apart and one more
    end = FAKE + 7 * GIB + 2 * (6 * 1024 + 128)
    assert call(ks=1024, c=cache(ks=end - 16)) == K.KQ_ERR_OVERLAP


def test_attention_refusals():
    q, out, work = FAKE + 7 * GIB, FAKE + 8 * GIB, FAKE + 9 * GIB

    def call(c=None, b=None, q=q, qs=512, heads=8, scale=0.125, window=0, sinks=0, out=out, os=512, work=work,
             size=1 << 20):
        return raw("mx_cache_attention", q, qs, heads, c or cache(), b or batch(), ctypes.c_float(scale), window, sinks,
                   out, os, work, size, None)

    for dim in (32, 96, 160, 192):
        assert call(cache(dim=dim), qs=2048, os=2048) == K.KQ_ERR_SHAPE, dim
    assert call(cache(pages=0)) == call(b=batch(rows=-1)) == call(b=batch(lengths=None)) == K.KQ_ERR_ARG
    assert call(heads=0) == call(window=-1) == call(sinks=-1) == call(size=-1) == K.KQ_ERR_ARG
    assert call(heads=7) == call(heads=4098) == call(window=(1 << 30) + 1) == call(sinks=(1 << 30) + 1) == K.KQ_ERR_SHAPE
    assert call(heads=4096, b=batch(rows=1 << 19), qs=1 << 18, os=1 << 18) == K.KQ_ERR_SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-31):
        assert call(scale=scale) == K.KQ_ERR_ARG, scale
    assert call(q=None) == call(out=None) == K.KQ_ERR_ARG
    assert call(q=q + 8) == call(out=out + 4) == call(work=work + 8) == K.KQ_ERR_ALIGN
    assert call(qs=511) == call(os=448) == K.KQ_ERR_SHAPE
    assert call(qs=516) == call(os=513) == K.KQ_ERR_ALIGN
    assert call(out=q + 64) == call(out=FAKE + 16) == call(work=FAKE + 3 * GIB) == call(work=out) == K.KQ_ERR_OVERLAP
    assert call(b=batch(row_start=out + 64)) == call(b=batch(page_table=work)) == K.KQ_ERR_OVERLAP
    assert call(b=batch(rows=0), q=None, out=None, work=None) == call(b=batch(seqs=0), q=None) == K.KQ_OK
    need = ctypes.c_int64(-1)

    def bytes_of(heads=8, c=None, b=None, window=0, to=ctypes.byref(need)):
        return raw("mx_cache_attention_workspace", heads, c or cache(), b or batch(), window, 0, to)

    assert bytes_of(to=None) == bytes_of(window=-1) == K.KQ_ERR_ARG
    assert bytes_of(heads=3) == bytes_of(c=cache(dim=96)) == K.KQ_ERR_SHAPE
    assert bytes_of(b=batch(rows=0)) == K.KQ_OK and need.value == 0


def test_binding_checks():
    torch = pytest.importorskip("torch")
    u8, i32 = torch.uint8, torch.int32
    c = K.mx_cache_new(2, 16, 2, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 2, 16, 32), (2, 2, 2, 16)] * 2
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    table, start, lengths = torch.zeros((1, 2), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(TypeError):  # host tensors
        K.mx_cache_write(x, x, c, table, start, lengths)
    with pytest.raises(TypeError):
        K.mx_cache_read(c, table, start, lengths, rows=3)
    with pytest.raises(TypeError):
        K.mx_gemv(torch.zeros((1, 32), dtype=torch.bfloat16), torch.zeros((4, 16), dtype=u8),
                  torch.zeros((4, 1), dtype=u8))
    with pytest.raises(ValueError):  # scales of another K
        K.mx_gemv(torch.zeros((1, 64), dtype=torch.bfloat16), torch.zeros((4, 32), dtype=u8),
                  torch.zeros((4, 1), dtype=u8))
    with pytest.raises(ValueError):
        K.mx_cache_new(2, 16, 2, 40, device="cpu")
    with pytest.raises(ValueError):  # buffers of two geometries
        K.mx_cache_read(c._replace(vs=c.vs[:1]), table, start, lengths, rows=3)


def test_compiled_host_side():
    """It is built from the library's sources, leaves what is not its call to
    the Python side, and minds its arguments' number."""
    torch = pytest.importorskip("torch")
    from mxfp4_act_quantizer_amd import build as B
    from mxfp4_act_quantizer_amd import _binding
    fast = _binding.load_serving()
    assert fast.source_hash == B.source_hash()
    x, w, s = torch.zeros((1, 64)).bfloat16(), torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.uint8)
    assert fast.gemv(x, w, s, None, True, 0) is None  # tensors of the CPU
    assert fast.gemv(1, "w", None, None, True, 0) is None
    cache = tuple(torch.zeros(n, dtype=torch.uint8) for n in ((1, 1, 16, 32), (1, 1, 2, 16)) * 2)
    i = torch.zeros((1, 1), dtype=torch.int32)
    assert fast.read(cache, i, i, i, 1, 0) is None and fast.read(None, i, i, i, 1, 0) is None
    assert fast.write(x, x, cache, i, i, i, None, 0) is None
    assert fast.attention(x, cache, i, i, i, None, 0, 0, None, 0) is None
    for f in (fast.gemv, fast.write, fast.read, fast.attention):
        with pytest.raises(TypeError):
            f(x)
