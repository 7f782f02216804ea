"""Host-side refusals of the paged cache's append and attention and of the
token log probabilities, and their struct layout: every check returns before
the first CUDA call, so no GPU is needed (placeholder addresses: none is
dereferenced)."""
import ctypes as C
import os
import subprocess

import pytest

import mtp_speculative_decoding_gb300 as mtp
from mtp_speculative_decoding_gb300 import build as mtp_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    mtp_build.build()


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_table=FAKE, stride_p=4 * 64 * 128, stride_h=64 * 128, stride_t=128,
             n_pages=10, page_size=64, max_pages=8, n_kv_heads=4, head_dim=128, kv_dtype=mtp.MTP_DTYPE_BF16, window=0, sink=0,
             rope_theta=1e4, pad_=0)
    d.update(kw)
    return mtp.KVCache(*[d[f] for f, _ in mtp.KVCache._fields_])


def append(c, B=2, M=3, kv_len=FAKE, n_new=None, k=FAKE, v=FAKE, dtype=mtp.MTP_DTYPE_BF16, sb=3 * 512, sm=512, sh=128, gain=None,
           eps=1e-6, ws=FAKE, nbytes=1 << 30):
    return mtp.lib().mtp_kv_append(C.byref(c) if c else None, B, M, kv_len, n_new, k, v, dtype, sb, sm, sh, gain, eps, ws, nbytes, None)


def attend(c, B=2, M=3, hq=8, kv_len=FAKE, n_new=None, q=FAKE, dtype=mtp.MTP_DTYPE_BF16, sb=3 * 1024, sm=1024, sh=128, gain=None,
           eps=1e-6, scale=0.0, out=FAKE, ws=FAKE, nbytes=1 << 30):
    return mtp.lib().mtp_paged_attention(C.byref(c) if c else None, B, M, hq, kv_len, n_new, q, dtype, sb, sm, sh, gain, eps, scale,
                                         out, ws, nbytes, None)


def logprobs(z=FAKE, dtype=mtp.MTP_DTYPE_BF16, rows=4, V=100, stride=100, tokens=FAKE, k=5, lp=FAKE, ent=FAKE, ids=FAKE, top=FAKE):
    return mtp.lib().mtp_token_logprobs(z, dtype, rows, V, stride, tokens, k, lp, ent, ids, top, None)


ARG, UNS, WS = mtp.MTP_ERR_ARG, mtp.MTP_ERR_UNSUPPORTED, mtp.MTP_ERR_WORKSPACE

BAD_CACHES = [
    (dict(k=None), ARG), (dict(v=FAKE + 8), ARG), (dict(page_table=None), ARG), (dict(page_table=FAKE + 2), ARG),
    (dict(n_pages=0), ARG), (dict(max_pages=0), ARG), (dict(n_kv_heads=0), ARG),
    (dict(head_dim=96), UNS), (dict(head_dim=1024), UNS), (dict(page_size=8), UNS), (dict(page_size=48), UNS),
    (dict(page_size=512), UNS), (dict(kv_dtype=7), UNS), (dict(max_pages=1 << 26), UNS),
    (dict(stride_t=120), ARG), (dict(stride_t=132), ARG), (dict(stride_h=-8), ARG), (dict(stride_p=4 * 64 * 128 + 4), ARG),
    (dict(window=-1), ARG), (dict(sink=4), ARG), (dict(rope_theta=-1.0), ARG), (dict(rope_theta=float("inf")), ARG),
    (dict(rope_theta=float("nan")), ARG),
    (dict(kv_dtype=mtp.MTP_DTYPE_E4M3), ARG),                                     # no scales
    (dict(kv_dtype=mtp.MTP_DTYPE_E4M3, k_scale=FAKE), ARG),
    (dict(kv_dtype=mtp.MTP_DTYPE_E4M3, k_scale=FAKE, v_scale=FAKE, stride_t=136), ARG),   # 8-bit rows: 16-byte strides
]


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=lambda x: str(x)[:60])
def test_bad_caches_are_refused(kw, code):
    c = cache(**kw)
    assert append(c) == code
    assert attend(c) == code


def test_bad_append_arguments():
    c = cache()
    assert append(None) == ARG
    for kw in (dict(B=0), dict(B=mtp.MTP_MAX_PAGED_BATCH + 1), dict(M=0), dict(M=mtp.MTP_MAX_APPEND_ROWS + 1), dict(kv_len=None),
               dict(kv_len=FAKE + 1), dict(n_new=FAKE + 2), dict(k=None), dict(v=None), dict(k=FAKE + 4), dict(sb=-8), dict(sm=516),
               dict(sh=100), dict(eps=-1.0), dict(eps=float("nan")), dict(gain=FAKE + 1)):
        assert append(c, **kw) == ARG, kw
    assert append(c, dtype=mtp.MTP_DTYPE_E4M3) == UNS
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(nbytes=255)):
        assert append(c, **kw) == WS, kw


def test_bad_attention_arguments():
    c = cache()
    assert attend(None) == ARG
    for kw in (dict(B=0), dict(B=mtp.MTP_MAX_PAGED_BATCH + 1), dict(M=0), dict(M=mtp.MTP_MAX_ATTN_ROWS + 1), dict(hq=0), dict(hq=6),
               dict(kv_len=None), dict(q=None), dict(q=FAKE + 8), dict(sb=-8), dict(sm=1028), dict(sh=4), dict(out=None),
               dict(out=FAKE + 8), dict(scale=-1.0), dict(scale=float("nan")), dict(eps=-1.0), dict(gain=FAKE + 2)):
        assert attend(c, **kw) == ARG, kw
    assert attend(c, hq=4 * 17) == UNS
    assert attend(c, dtype=mtp.MTP_DTYPE_E4M3) == UNS


def test_bad_logprob_arguments():
    for kw in (dict(z=None), dict(z=FAKE + 1), dict(rows=0), dict(rows=17 * mtp.MTP_MAX_VERIFY_BATCH + 1), dict(V=0), dict(stride=99),
               dict(k=-1), dict(k=mtp.MTP_MAX_TOP + 1), dict(tokens=FAKE + 2), dict(lp=FAKE + 1), dict(ent=FAKE + 3), dict(ids=FAKE + 1),
               dict(top=FAKE + 2), dict(dtype=mtp.MTP_DTYPE_F32, z=FAKE + 2)):
        assert logprobs(**kw) == ARG, kw
    assert logprobs(dtype=mtp.MTP_DTYPE_E4M3) == UNS


def test_workspace_size_needs_no_gpu():
    c = cache()
    n = mtp.kv_workspace_size(c, 2, 3, 8)
    assert n % 256 == 0 and n > 256
    assert mtp.kv_workspace_size(c, 2, 4096, 8) >= 256          # an append's
    for kw in (dict(B=0), dict(M=0), dict(B=mtp.MTP_MAX_PAGED_BATCH + 1), dict(n_q_heads=6)):
        with pytest.raises(mtp.MTPError):
            mtp.kv_workspace_size(c, **{**dict(B=2, M=3, n_q_heads=8), **kw})
    with pytest.raises(mtp.MTPError):
        mtp.kv_workspace_size(cache(head_dim=96), 2, 3, 8)


def test_cache_struct_matches_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "mtp.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(mtp_kv_cache));']
    lines += ['printf("%s %%zu\\n", offsetof(mtp_kv_cache, %s));' % (f, f) for f, _ in mtp.KVCache._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    assert int(got.pop("size")) == C.sizeof(mtp.KVCache)
    assert {f: int(v) for f, v in got.items()} == {f: getattr(mtp.KVCache, f).offset for f, _ in mtp.KVCache._fields_}


def test_binding_refuses_cpu_tensors():
    import torch
    k = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError):
        mtp.make_kv_cache(k, k, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mtp.token_logprobs(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32), torch.zeros(2))
