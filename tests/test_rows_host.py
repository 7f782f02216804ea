"""Host-side refusals of the attention of prompts and of shared prefixes and of
the rotation by several positions: every check returns before the first CUDA
call, so no GPU is needed (placeholder addresses: none is dereferenced)."""
import ctypes as C

import pytest

import mtp_speculative_decoding_gb300 as mtp
from mtp_speculative_decoding_gb300 import build as mtp_build
from test_paged_host import ARG, BAD_CACHES, FAKE, UNS, WS, cache


@pytest.fixture(scope="module", autouse=True)
def _built():
    mtp_build.build()


def prompt(c, B=2, T=100, hq=8, kv_len=FAKE, start=FAKE, q=FAKE, dtype=mtp.MTP_DTYPE_BF16, sm=1024, sh=128, gain=None, eps=1e-6,
           scale=0.0, out=FAKE, ws=FAKE, nbytes=1 << 40):
    return mtp.lib().mtp_prompt_attention(C.byref(c) if c else None, B, T, hq, kv_len, start, q, dtype, sm, sh, gain, eps, scale, out, ws,
                                          nbytes, None)


def prefix(c, B=2, M=3, hq=8, kv_len=FAKE, n_new=None, groups=1, start=FAKE, length=FAKE, q=FAKE, dtype=mtp.MTP_DTYPE_BF16, sb=3 * 1024,
           sm=1024, sh=128, gain=None, eps=1e-6, scale=0.0, out=FAKE, ws=FAKE, nbytes=1 << 40):
    return mtp.lib().mtp_prefix_attention(C.byref(c) if c else None, B, M, hq, kv_len, n_new, groups, start, length, q, dtype, sb, sm, sh,
                                          gain, eps, scale, out, ws, nbytes, None)


def rotate(rows=5, axes=3, pos=FAKE, sections=(24, 20, 20), inter=0, theta=1e4, hd=128, dtype=mtp.MTP_DTYPE_BF16, q=FAKE, hq=8, qm=1024,
           qh=128, k=FAKE, hk=2, km=256, kh=128, qn=None, kn=None, eps=1e-6, oq=FAKE, oqm=1024, oqh=128, ok=FAKE, okm=256, okh=128):
    sec = (C.c_int32 * len(sections))(*sections) if sections is not None else None
    return mtp.lib().mtp_rotate_axes(rows, axes, pos, sec, inter, theta, hd, dtype, q, hq, qm, qh, k, hk, km, kh, qn, kn, eps, oq, oqm, oqh,
                                     ok, okm, okh, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=lambda x: str(x)[:60])
def test_bad_caches_are_refused(kw, code):
    assert prompt(cache(**kw)) == code
    assert prefix(cache(**kw)) == code


COMMON = (dict(B=0), dict(B=mtp.MTP_MAX_PAGED_BATCH + 1), dict(hq=0), dict(hq=6), dict(kv_len=None), dict(kv_len=FAKE + 2), dict(q=None),
          dict(q=FAKE + 8), dict(sm=1028), dict(sh=4), dict(out=None), dict(out=FAKE + 8), dict(scale=-1.0), dict(scale=float("nan")),
          dict(scale=float("inf")), dict(eps=-1.0), dict(gain=FAKE + 2))


def test_bad_prompt_arguments():
    c = cache()
    assert prompt(None) == ARG
    for kw in COMMON + (dict(T=0), dict(T=mtp.MTP_MAX_PROMPT_ROWS + 1), dict(start=None), dict(start=FAKE + 1)):
        assert prompt(c, **kw) == ARG, kw
    assert prompt(c, hq=4 * 17) == UNS
    assert prompt(c, dtype=mtp.MTP_DTYPE_E4M3) == UNS
    assert prompt(cache(n_kv_heads=1024), T=mtp.MTP_MAX_PROMPT_ROWS, hq=2048) == UNS      # 2^31 rows of heads
    need = mtp.prompt_workspace_size(c, 2, 100, 8)
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(nbytes=need - 1)):
        assert prompt(c, **kw) == WS, kw


def test_bad_prefix_arguments():
    c = cache()
    assert prefix(None) == ARG
    for kw in COMMON + (dict(M=0), dict(M=mtp.MTP_MAX_ATTN_ROWS + 1), dict(n_new=FAKE + 1), dict(sb=-8), dict(groups=-1), dict(groups=3),
                        dict(start=None), dict(length=None), dict(start=FAKE + 1), dict(length=FAKE + 2)):
        assert prefix(c, **kw) == ARG, kw
    assert prefix(c, hq=4 * 17) == UNS
    assert prefix(c, dtype=mtp.MTP_DTYPE_E4M3) == UNS
    assert prefix(cache(window=128)) == UNS
    need = mtp.prefix_workspace_size(c, 2, 3, 8)
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(nbytes=need - 1)):
        assert prefix(c, **kw) == WS, kw


def test_bad_rotate_arguments():
    for kw in (dict(rows=0), dict(rows=mtp.MTP_MAX_PROMPT_ROWS + 1), dict(axes=0), dict(axes=5, sections=(8,) * 5), dict(sections=None),
               dict(pos=None), dict(pos=FAKE + 2), dict(theta=0.0), dict(theta=-1.0), dict(theta=float("inf")), dict(theta=float("nan")),
               dict(eps=-1.0), dict(sections=(24, -8, 48)), dict(sections=(0, 0, 0)), dict(sections=(40, 20, 20)), dict(q=None),
               dict(q=FAKE + 8), dict(hq=0), dict(hk=0), dict(qm=1028), dict(qh=-8), dict(km=4), dict(k=FAKE + 4), dict(qn=FAKE + 1),
               dict(kn=FAKE + 3), dict(oq=None), dict(oq=FAKE + 8), dict(ok=None), dict(okh=12), dict(oqm=1020)):
        assert rotate(**kw) == ARG, kw
    assert rotate(hd=96, sections=(16, 16, 16)) == UNS
    assert rotate(dtype=mtp.MTP_DTYPE_E4M3) == UNS
    assert rotate(sections=(20, 20, 20)) == UNS                       # 60 pairs
    assert rotate(rows=mtp.MTP_MAX_PROMPT_ROWS, hq=2048, qm=2048 * 128) == UNS


def test_workspace_sizes_need_no_gpu():
    c = cache()
    for size, ok, bad in ((mtp.prompt_workspace_size, (2, 100, 8), ((0, 100, 8), (2, 0, 8), (2, mtp.MTP_MAX_PROMPT_ROWS + 1, 8), (2, 100, 6))),
                          (mtp.prefix_workspace_size, (2, 3, 8), ((0, 3, 8), (2, 65, 8), (mtp.MTP_MAX_PAGED_BATCH + 1, 3, 8), (2, 3, 6)))):
        n = size(c, *ok)
        assert n >= 256 and n % 256 == 0
        for args in bad:
            with pytest.raises(mtp.MTPError):
                size(c, *args)
        with pytest.raises(mtp.MTPError):
            size(cache(head_dim=96), *ok)


def test_binding_refuses_wrong_shapes():
    import torch
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)   # noqa: E731
    c = cache()
    with pytest.raises(ValueError):
        mtp.prompt_attention(c, z(5, 8, 64), i(3), i(2), z(5, 8, 64), z(256))
    with pytest.raises(ValueError):
        mtp.prompt_attention(c, z(5, 8, 128), i(2), i(2), z(5, 8, 128), z(256))       # row_start: [B + 1]
    with pytest.raises(ValueError):
        mtp.prefix_attention(c, z(2, 3, 8, 64), i(2), i(2), i(1), z(2, 3, 8, 64), z(256))
    with pytest.raises(ValueError):
        mtp.prefix_attention(c, z(2, 3, 8, 128), i(2), i(3), i(1), z(2, 3, 8, 128), z(256))   # group_start: [groups + 1]
    q, k = z(5, 8, 128), z(5, 2, 128)
    for args in ((q[0], k, i(3, 5), (24, 20, 20), 1e4, q[0], k), (q, k[:4], i(3, 5), (24, 20, 20), 1e4, q, k[:4]),
                 (q, k, i(3, 5), (24, 20, 20), 1e4, q, None), (q, k, i(2, 5), (24, 20, 20), 1e4, q, k),
                 (q, k, i(3, 5), (24, 20, 20), 1e4, q[:4], k), (q, k.half(), i(3, 5), (24, 20, 20), 1e4, q, k.half())):
        with pytest.raises(ValueError):
            mtp.rotate_axes(*args)


def test_more_cached_positions_than_the_plan_counts_are_refused():
    c = cache(max_pages=0x7FFFFF00 // 16, page_size=16)
    for size, call, most in ((mtp.prefix_workspace_size, prefix, 127),):
        assert size(c, most, 3, 8) > 0
        with pytest.raises(mtp.MTPError):
            size(c, most + 1, 3, 8)
        assert call(c, B=most + 1) == UNS
