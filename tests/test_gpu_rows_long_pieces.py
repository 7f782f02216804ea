"""One worker's piece of an item may take longer than the limit of a single wait:
the wait for the next item's turn counts the piece's tiles.

The library is linked here with a limit of 20 ms in the place of a second, and
the pieces take longer than that."""
import ctypes as C
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import mtp_speculative_decoding_gb300 as m
    from mtp_speculative_decoding_gb300 import build as b
    b.build()
    d = tmp_path_factory.mktemp("limit")
    with open(os.path.join(b.CSRC, "paged_api.cu")) as f:
        text = f.read()
    limit = "kWaitLimitNs = 1000000000ull"
    assert text.count(limit) == 1
    src, so = d / "paged_api.cu", d / "libmtp_limit.so"
    src.write_text(text.replace(limit, "kWaitLimitNs = 20000000ull"))
    objects = [os.path.join(b.BUILD, n + ".o") for n, _, _ in b.UNITS if n != "paged_api"]
    r = subprocess.run([b._nvcc()] + b._flags() + ["-shared", "-cudart", "shared", str(src)] + objects + ["-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = C.CDLL(str(so))
    for name in ("mtp_prompt_workspace_size", "mtp_prompt_attention"):
        f = getattr(L, name)
        f.argtypes, f.restype = getattr(m.lib(), name).argtypes, getattr(m.lib(), name).restype
    return L


@pytest.mark.parametrize("kv,hd,pages", [("bf16", 64, 80000), ("bf16", 256, 40000), ("e4m3", 128, 60000)])
def test_pieces_longer_than_a_waits_limit(lib, kv, hd, pages):
    """More items than workers, each of them many tiles long (every page of the
    table is the same one): keys of zero weigh all positions alike, so the result
    is the page's mean value, exactly."""
    import mtp_speculative_decoding_gb300 as m
    ps, hkv = 256, 200
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    k = torch.zeros((1, hkv, ps, hd), device="cuda").to(dt)
    v = torch.exp2(torch.arange(hd, device="cuda") % 5).expand(1, hkv, ps, hd).to(dt).contiguous()
    sc = torch.ones((1, hkv), device="cuda") if kv == "e4m3" else None
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    h = m.make_kv_cache(k, v, table, sc, sc, rope_theta=1e6)
    q = torch.ones((1, hkv, hd), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    at = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([pages * ps - 1], dtype=torch.int32, device="cuda")
    ws = m.alloc_workspace(lib.mtp_prompt_workspace_size(C.byref(h), 1, 1, hkv))
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    rc = lib.mtp_prompt_attention(C.byref(h), 1, 1, hkv, lens.data_ptr(), at.data_ptr(), q.data_ptr(), m.MTP_DTYPE_BF16, q.stride(0), q.stride(1),
                                  None, 1e-6, 0.0, out.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    ev[1].record()
    assert rc == m.MTP_OK and m.last_error(ws) == m.MTP_OK
    took = ev[0].elapsed_time(ev[1])
    assert took > 40, f"{took} ms: no piece was longer than the limit"
    # (sums of up to 2^25 terms that are multiples of 128: exact)
    assert torch.equal(out, v[:, :, 0].to(torch.bfloat16))
