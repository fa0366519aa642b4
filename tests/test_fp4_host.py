"""CPU checks of the 4-bit cache's entry points: refusals on the host before any HIP
call, shapes in the binding, and the plain form the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd.binding import PagedKv
from fp4_ref import MAGNITUDES, held, quantise

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
FAKE = 0x10000      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return df2.load()


def kv(**kw):
    d = dict(k_cache=FAKE, v_cache=FAKE, block_table=FAKE, ctx_len=FAKE, tok_start=FAKE, page_stride=2 * 16 * 68,
             table_stride=8, B=2, N=5, Hq=8, Hkv=2, D=128, page_size=16, num_pages=10, table_width=8, dtype=1)
    d.update(kw)
    return PagedKv(*[d[n] for n, _ in PagedKv._fields_])


BAD_KV = [
    (dict(dtype=7), EINVAL, "dtype"), (dict(B=-1), EINVAL, "B and N"), (dict(N=-1), EINVAL, "B and N"),
    (dict(Hq=7), EINVAL, "Hq"), (dict(Hkv=0), EINVAL, "Hq"), (dict(D=96), EUNSUPPORTED, "D must"),
    (dict(page_size=24), EUNSUPPORTED, "page_size"), (dict(page_size=8), EUNSUPPORTED, "at least 16"),
    (dict(page_size=1), EUNSUPPORTED, "at least 16"), (dict(num_pages=0), EINVAL, "num_pages"),
    (dict(table_width=0), EINVAL, "table_width"), (dict(table_stride=7), EINVAL, "table_width"),
    (dict(table_width=1 << 27, table_stride=1 << 27), EUNSUPPORTED, "2^30"), (dict(N=1 << 30), EUNSUPPORTED, "N * Hq"),
    (dict(page_stride=2175), EINVAL, "page_stride"), (dict(page_stride=2184), EINVAL, "page_stride"),
    (dict(k_cache=None), EINVAL, "NULL"), (dict(tok_start=None), EINVAL, "NULL"), (dict(v_cache=FAKE + 8), EINVAL, "aligned"),
    (dict(ctx_len=FAKE + 2), EINVAL, "aligned"),
]


def attend(lib, k, q=FAKE, q_stride=1024, scale=0.1, causal=1, window=0, max_len=64, out=FAKE + (1 << 20), out_stride=1024,
           ws=None, n=0):
    return lib.dflash2_paged_attention_fp4(ctypes.byref(k) if k is not None else None, q, q_stride, scale, causal, window,
                                           max_len, out, out_stride, ws, n, None)


def append(lib, k, q=FAKE, q_stride=1024, kk=FAKE, k_stride=256, v=FAKE, v_stride=256, qn=None, kn=None, eps=1e-6,
           freq=FAKE, rot=128, out=FAKE, out_stride=1024):
    return lib.dflash2_kv_append_fp4(ctypes.byref(k) if k is not None else None, q, q_stride, kk, k_stride, v, v_stride,
                                     qn, kn, eps, freq, rot, 0, out, out_stride, None)


@pytest.mark.parametrize("change,status,msg", BAD_KV)
def test_cache_descriptor_is_checked(lib, change, status, msg):
    for call in (attend, append):
        assert call(lib, kv(**change)) == status
        assert msg in lib.dflash2_last_error().decode()


def test_attention_refusals(lib):
    assert attend(lib, None) == EINVAL
    for kw, msg in ((dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
                    (dict(window=-1), "window"), (dict(max_len=-1), "max_len"), (dict(q=None), "NULL"),
                    (dict(out=None), "NULL"), (dict(q=FAKE + 4), "aligned"), (dict(q_stride=1020), "stride"),
                    (dict(out_stride=1028), "stride"), (dict(out=FAKE), "overlap")):
        ws = dict(ws=FAKE, n=1 << 30)
        assert attend(lib, kv(), **ws, **kw) == EINVAL, kw
        assert msg in lib.dflash2_last_error().decode()
    assert attend(lib, kv(N=0, k_cache=None), q=None) == OK
    assert attend(lib, kv(B=0), q=None) == OK


def test_attention_workspace(lib):
    f = lib.dflash2_paged_attention_fp4_workspace
    long = kv(table_width=4096, table_stride=4096)
    need = f(ctypes.byref(long), 0)
    assert need > 0 and need % 4 == 0
    assert f(ctypes.byref(kv(N=0)), 16) == 0 and f(ctypes.byref(kv(D=77)), 0) == 0 and f(None, 0) == 0
    assert attend(lib, long, max_len=0, ws=None, n=need) == EINVAL
    assert str(need) in lib.dflash2_last_error().decode()
    assert attend(lib, long, max_len=0, ws=FAKE, n=need - 1) == EINVAL
    assert attend(lib, long, max_len=0, ws=FAKE + 4, n=need) == EINVAL


def test_append_refusals(lib):
    assert append(lib, None) == EINVAL
    for kw, status, msg in ((dict(rot=24), EUNSUPPORTED, "rot"), (dict(rot=144), EUNSUPPORTED, "rot"), (dict(eps=-1.0), EINVAL, "eps"),
                            (dict(eps=float("nan")), EINVAL, "eps"), (dict(kk=None), EINVAL, "NULL"), (dict(v=None), EINVAL, "NULL"),
                            (dict(freq=None), EINVAL, "NULL"), (dict(out=None), EINVAL, "together"),
                            (dict(q=None, out=None, qn=FAKE), EINVAL, "q_norm"), (dict(k_stride=255), EINVAL, "stride"),
                            (dict(q=FAKE + 2), EINVAL, "aligned"), (dict(qn=FAKE + 8), EINVAL, "aligned"),
                            (dict(freq=FAKE + 4), EINVAL, "aligned"), (dict(out_stride=2048), EINVAL, "same stride")):
        assert append(lib, kv(), **kw) == status, kw
        assert msg in lib.dflash2_last_error().decode(), kw
    assert append(lib, kv(N=0)) == OK


def test_unpack_refusals(lib):
    def call(k, out_k=FAKE + (1 << 30), out_v=FAKE + (1 << 31)):
        return lib.dflash2_kv_unpack_fp4(ctypes.byref(k) if k is not None else None, out_k, out_v, None)
    far = dict(k_cache=FAKE, v_cache=FAKE + (1 << 29), block_table=None, ctx_len=None, tok_start=None, B=0, N=0)
    assert call(None) == EINVAL
    for change, kw, status, msg in ((dict(D=96), {}, EUNSUPPORTED, "D must"), (dict(page_size=8), {}, EUNSUPPORTED, "at least 16"),
                                    (dict(k_cache=None), {}, EINVAL, "NULL"), ({}, dict(out_v=None), EINVAL, "NULL"),
                                    (dict(v_cache=FAKE + 8), {}, EINVAL, "aligned"), ({}, dict(out_k=FAKE + 4), EINVAL, "aligned"),
                                    ({}, dict(out_k=FAKE + 1024), EINVAL, "cache"), ({}, dict(out_v=FAKE + (1 << 30) + 64), EINVAL, "each other"),
                                    (dict(num_pages=(1 << 31) - 1), {}, EUNSUPPORTED, "2^34")):
        assert call(kv(**dict(far, **change)), **kw) == status, (change, kw)
        assert msg in lib.dflash2_last_error().decode()


def test_binding_refuses_bad_shapes():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc, vc = df2.fp4_cache(4, 2, 16, 128, device="cpu")
    assert kc.shape == (4, 2, 16 * 68) and df2.fp4_page_bytes(16, 128) == 16 * 68
    q, k = torch.zeros((5, 8, 128)), torch.zeros((5, 2, 128))
    where = (i(2, 3), i(2), i(3))
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.paged_attention_fp4(q, kc, vc, *where)
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.kv_append_fp4(k, k, kc, vc, *where)
    with pytest.raises(ValueError, match="uint8"):
        df2.paged_attention_fp4(q, kc.int(), vc.int(), *where)
    with pytest.raises(ValueError, match="no rows of head size"):
        df2.paged_attention_fp4(q, kc[..., :100], vc[..., :100], *where)
    with pytest.raises(ValueError, match=r"\[N, Hq, D\]"):
        df2.paged_attention_fp4(q[0], kc, vc, *where)
    with pytest.raises(ValueError, match=r"\[N, Hkv, D\]"):
        df2.kv_append_fp4(k[0], k[0], kc, vc, *where)
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.kv_unpack_fp4(kc, vc, 128)
    with pytest.raises(ValueError, match="32 bits"):
        df2.paged_attention_fp4(q, kc, vc, *where, window=2**32)


def test_plain_form():
    """Every code under its scale is its own nearest value; a block's largest decides."""
    x = np.zeros((9, 64))
    for row, top in enumerate((6.0, 7.0, 7.0000001, 3.5, 3.4999, 12.0, 0.0, 2.0 ** -121, 2.0 ** 127)):
        x[row, 3] = -top
        x[row, 40] = top
    codes, scales, bad = quantise(x)
    assert scales[:, 0].tolist() == [127, 127, 128, 126, 126, 128, 7, 7, 247] and not bad.any()
    full = np.concatenate((codes.reshape(1, 1, -1), scales.reshape(1, 1, -1)), -1)
    got = held(torch.from_numpy(full), 9, 64)[0, 0].numpy()
    assert got[:, 40].tolist() == [6.0, 6.0, 8.0, 3.0, 3.0, 12.0, 0.0, 2.0 ** -121, 6 * 2.0 ** 120]
    assert (got[:, 3] == -got[:, 40]).all()
    every = np.concatenate((MAGNITUDES, -MAGNITUDES, MAGNITUDES, -MAGNITUDES))[None]
    c, s, _ = quantise(every * 2.0 ** 20)
    back = held(torch.from_numpy(np.concatenate((c, s), -1).reshape(1, 1, -1)), 1, 32)
    assert np.array_equal(back[0, 0, 0].numpy(), every[0] * 2.0 ** 20)
