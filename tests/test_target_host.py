"""CPU checks of the target-side entry points: every refusal happens on the
host before any HIP call, and the binding checks shapes before pointers."""
import ctypes

import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd.binding import PagedKv, VerifyDims
from target_ref import append_ref, attention_ref, paged_case, verify_ref

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
FAKE = 0x10000      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return df2.load()


def kv(**kw):
    d = dict(k_cache=FAKE, v_cache=FAKE, block_table=FAKE, ctx_len=FAKE, tok_start=FAKE, page_stride=2 * 16 * 128,
             table_stride=8, B=2, N=5, Hq=8, Hkv=2, D=128, page_size=16, num_pages=10, table_width=8, dtype=1)
    d.update(kw)
    return PagedKv(*[d[n] for n, _ in PagedKv._fields_])


BAD_KV = [
    (dict(dtype=7), EINVAL, "dtype"), (dict(B=-1), EINVAL, "B and N"), (dict(N=-1), EINVAL, "B and N"),
    (dict(Hq=7), EINVAL, "Hq"), (dict(Hkv=0), EINVAL, "Hq"), (dict(D=96), EUNSUPPORTED, "D must"),
    (dict(page_size=24), EUNSUPPORTED, "page_size"), (dict(page_size=0), EUNSUPPORTED, "page_size"),
    (dict(num_pages=0), EINVAL, "num_pages"), (dict(table_width=0), EINVAL, "table_width"),
    (dict(table_stride=7), EINVAL, "table_width"), (dict(table_width=1 << 27, table_stride=1 << 27), EUNSUPPORTED, "2^30"),
    (dict(N=1 << 30), EUNSUPPORTED, "N * Hq"), (dict(page_stride=4095), EINVAL, "page_stride"),
    (dict(page_stride=4097), EINVAL, "page_stride"), (dict(k_cache=None), EINVAL, "NULL"),
    (dict(tok_start=None), EINVAL, "NULL"), (dict(v_cache=FAKE + 8), EINVAL, "aligned"),
    (dict(ctx_len=FAKE + 2), EINVAL, "aligned"),
]


def attend(lib, k, q=FAKE, q_stride=1024, scale=0.1, causal=1, window=0, max_len=64, out=FAKE, out_stride=1024,
           ws=None, n=0):
    return lib.dflash2_paged_attention(ctypes.byref(k) if k is not None else None, q, q_stride, scale, causal, window,
                                       max_len, out, out_stride, ws, n, None)


def append(lib, k, q=FAKE, q_stride=1024, kk=FAKE, k_stride=256, v=FAKE, v_stride=256, qn=None, kn=None, eps=1e-6,
           freq=FAKE, rot=128, out=FAKE, out_stride=1024):
    return lib.dflash2_kv_append(ctypes.byref(k) if k is not None else None, q, q_stride, kk, k_stride, v, v_stride,
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
                    (dict(out_stride=1028), "stride")):
        assert attend(lib, kv(), **kw) == EINVAL, kw
        assert msg in lib.dflash2_last_error().decode()
    # nothing to do: nothing is looked at beyond the sizes
    assert attend(lib, kv(N=0, k_cache=None), q=None) == OK
    assert attend(lib, kv(B=0), q=None) == OK


def test_attention_workspace(lib):
    long = kv(table_width=4096, table_stride=4096)
    need = lib.dflash2_paged_attention_workspace(ctypes.byref(long), 0)
    assert need > 0 and need % 4 == 0
    one = kv(B=1, N=1, Hq=1, Hkv=1, page_stride=16 * 128)
    assert lib.dflash2_paged_attention_workspace(ctypes.byref(one), 1) < need
    assert lib.dflash2_paged_attention_workspace(ctypes.byref(kv(N=0)), 16) == 0
    assert lib.dflash2_paged_attention_workspace(ctypes.byref(kv(D=77)), 0) == 0
    assert lib.dflash2_paged_attention_workspace(None, 0) == 0
    assert attend(lib, long, max_len=0, ws=None, n=need) == EINVAL
    assert str(need) in lib.dflash2_last_error().decode()
    assert attend(lib, long, max_len=0, ws=FAKE, n=need - 1) == EINVAL
    assert attend(lib, long, max_len=0, ws=FAKE + 4, n=need) == EINVAL


def test_append_refusals(lib):
    assert append(lib, None) == EINVAL
    for kw, status, msg in ((dict(rot=24), EUNSUPPORTED, "rot"), (dict(rot=144), EUNSUPPORTED, "rot"),
                            (dict(rot=-16), EUNSUPPORTED, "rot"), (dict(eps=-1.0), EINVAL, "eps"),
                            (dict(eps=float("nan")), EINVAL, "eps"), (dict(kk=None), EINVAL, "NULL"),
                            (dict(v=None), EINVAL, "NULL"), (dict(freq=None), EINVAL, "NULL"),
                            (dict(out=None), EINVAL, "together"), (dict(q=None), EINVAL, "together"),
                            (dict(q=None, out=None, qn=FAKE), EINVAL, "q_norm"), (dict(k_stride=255), EINVAL, "stride"),
                            (dict(v_stride=128), EINVAL, "stride"), (dict(q=FAKE + 2), EINVAL, "aligned"),
                            (dict(qn=FAKE + 8), EINVAL, "aligned"), (dict(freq=FAKE + 4), EINVAL, "aligned"),
                            (dict(out_stride=2048), EINVAL, "same stride")):
        assert append(lib, kv(), **kw) == status, kw
        assert msg in lib.dflash2_last_error().decode(), kw
    assert append(lib, kv(N=0)) == OK


def test_verify_refusals(lib):
    def call(dims, t=FAKE, path=FAKE, cand=FAKE, prob=FAKE, nd=None, tau=1.0, u=FAKE, o=(FAKE, FAKE, FAKE), ws=FAKE,
             n=1 << 30):
        return lib.dflash2_verify(ctypes.byref(dims) if dims is not None else None, t, path, cand, prob, nd, tau, u,
                                  o[0], o[1], o[2], ws, n, None)

    good = VerifyDims(2, 7, 1000, 16, 1, 0)
    assert call(None) == EINVAL
    for dims, status, msg in (((2, 7, 1000, 16, 5, 0), EINVAL, "dtype"), ((2, 7, 1000, 16, 1, 2), EINVAL, "kind"),
                              ((-1, 7, 1000, 16, 1, 0), EINVAL, "B < 0"), ((2, 0, 1000, 16, 1, 0), EINVAL, "P must"),
                              ((2, 65, 1000, 16, 1, 0), EINVAL, "P must"), ((2, 7, 0, 16, 1, 0), EINVAL, "V < 1"),
                              ((2, 7, (1 << 29) + 1, 16, 1, 0), EUNSUPPORTED, "V above"),
                              ((2, 7, 10, 11, 1, 0), EINVAL, "K must"), ((2, 7, 1000, 65, 1, 0), EINVAL, "K must"),
                              ((1 << 24, 7, 1000, 16, 1, 0), EUNSUPPORTED, "too large")):
        assert call(VerifyDims(*dims)) == status, dims
        assert msg in lib.dflash2_last_error().decode()
        assert lib.dflash2_verify_workspace(ctypes.byref(VerifyDims(*dims))) == 0
    for tau in (-1.0, float("nan"), float("inf"), 1e-39, 2e30):
        assert call(good, tau=tau) == EINVAL
        assert b"temperature" in lib.dflash2_last_error()
    for kw in (dict(t=None), dict(path=None), dict(cand=None), dict(prob=None), dict(u=None), dict(o=(None, FAKE, FAKE)),
               dict(t=FAKE + 1), dict(u=FAKE + 2), dict(nd=FAKE + 2), dict(ws=None), dict(n=16), dict(ws=FAKE + 8)):
        assert call(good, **kw) == EINVAL, kw
    assert call(VerifyDims(0, 7, 1000, 16, 1, 0), t=None) == OK
    assert lib.dflash2_verify_workspace(ctypes.byref(VerifyDims(0, 7, 1000, 16, 1, 0))) == 0


def test_draft_rows_refusals(lib):
    f = lib.dflash2_draft_rows
    assert f(FAKE, FAKE, FAKE, 0, 3, 4, 1.0, FAKE, None) == OK
    for args in ((FAKE, FAKE, FAKE, -1, 3, 4, 1.0, FAKE), (FAKE, FAKE, FAKE, 2, 0, 4, 1.0, FAKE),
                 (FAKE, FAKE, FAKE, 2, 65, 4, 1.0, FAKE), (FAKE, FAKE, FAKE, 2, 3, 65, 1.0, FAKE),
                 (FAKE, FAKE, FAKE, 2, 3, 4, 0.0, FAKE), (None, FAKE, FAKE, 2, 3, 4, 1.0, FAKE),
                 (FAKE, FAKE, None, 2, 3, 4, 1.0, FAKE), (FAKE, FAKE + 2, FAKE, 2, 3, 4, 1.0, FAKE)):
        assert f(*args, None) == EINVAL, args


def test_select_sample_rows_refusals(lib):
    from draft_selection_topk16_amd.binding import Dims
    d = Dims(1, 7, 32000, 1024, 256, 1)
    f = lib.dflash2_select_sample_rows

    def call(out_cand=FAKE, out_rows=FAKE, tau=1.0, u=FAKE):
        return f(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 16, tau, u, FAKE, FAKE, FAKE, out_cand, out_rows,
                 None)
    for kw in (dict(out_cand=None), dict(out_rows=None), dict(out_cand=FAKE + 2), dict(out_rows=FAKE + 1),
               dict(tau=0.0), dict(u=None)):
        assert call(**kw) == EINVAL, kw


def test_binding_refuses_bad_shapes():
    c = paged_case(1, torch.bfloat16, 64, 4, 2, 16, [3, 2], [5, 0], device="cpu")
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    args = (c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.paged_attention(c["q"], *args)
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.kv_append(k, k, *args)
    with pytest.raises(ValueError, match="one dtype"):
        df2.paged_attention(c["q"], c["k_cache"], c["v_cache"].float(), *args[2:])
    x = torch.zeros((2, 4, 50))
    path = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="kind"):
        df2.verify(x, path, kind="scores")
    with pytest.raises(ValueError, match="path"):
        df2.verify(x, path[:, :2])
    with pytest.raises(ValueError, match="prob"):
        df2.verify(x, path, path[..., None].expand(2, 3, 4), torch.zeros((2, 3, 5)), torch.zeros((2, 4)))
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.verify(x, path, temperature=0.0)
    with pytest.raises(ValueError, match="sampling"):
        df2.PreparedSelect(*([None] * 6), 16, rows=True)


def test_plain_forms_agree_with_torch():
    """The fp64 forms against another writing of the same formulas."""
    c = paged_case(2, torch.float32, 64, 4, 2, 16, [3], [20], device="cpu")
    out, bound = attention_ref(c, 0.125)
    ids = c["table"][0].long()
    kk = c["k_cache"][ids].transpose(0, 1).reshape(2, -1, 64)[:, :23].double()
    vv = c["v_cache"][ids].transpose(0, 1).reshape(2, -1, 64)[:, :23].double()
    mask = torch.arange(23) <= 20 + torch.arange(3)[:, None]
    for h in range(4):
        s = (c["q"][:, h].double() @ kk[h // 2].T * 0.125).masked_fill(~mask, -float("inf"))
        assert torch.allclose(out[:, h], torch.softmax(s, -1) @ vv[h // 2], rtol=1e-12)
    assert float(bound.max()) < 1e-3
    # a turn keeps lengths, and turning by p + r after norming equals turning twice
    x = torch.randn(2, 64).numpy()
    f = df2.rope_freqs(64, 1e4).numpy()
    for inter in (False, True):
        once, _ = append_ref(x, None, 0.0, f, 11, inter)
        twice, _ = append_ref(append_ref(x, None, 0.0, f, 4, inter)[0], None, 0.0, f, 7, inter)
        assert abs(once - twice).max() < 1e-12
    # greedy verification is sampling from one-hot rows
    x = torch.randn(3, 4, 20)
    path = x[:, :3].argmax(-1).to(torch.int32)
    path[1, 1] += 1
    tok, cnt, _, _ = verify_ref(x, path, None, None, None, 0.0)
    assert cnt.tolist() == [4, 2, 4] and tok[1].tolist()[2:] == [-1, -1]
