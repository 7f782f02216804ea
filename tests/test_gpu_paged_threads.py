"""Calls of different sizes from two host threads at once: what one call asks
of the runtime for its kernel does not disturb the other's launch."""
import ctypes as C
import threading

import pytest
import torch

import paged_common as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def together(calls, times):
    """Every call's worst return code over `times` turns, each in a thread of its own."""
    codes = [0] * len(calls)
    gate = threading.Barrier(len(calls))

    def loop(i):
        gate.wait()
        for _ in range(times):
            codes[i] = min(codes[i], calls[i]())

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return codes


def test_attention_of_two_head_sizes():
    import mtp_speculative_decoding_gb300 as m
    calls, keep = [], []
    for hd, s in ((512, torch.cuda.Stream()), (256, torch.cuda.Stream())):
        pool = pc.Pool(1, 2, 16, 1, hd, "f32", seed=1)
        pool.fill([17], seed=2)
        h = pool.handle()
        q = torch.randn(1, 1, 2, hd, device="cuda")
        out = torch.zeros_like(q)
        ln = torch.tensor([16], dtype=torch.int32, device="cuda")
        size = m.kv_workspace_size(h, 1, 1, 2)
        ws = m.alloc_workspace(size)
        keep.append((pool, h, q, out, ln, ws, s))
        args = (C.byref(h), 1, 1, 2, ln.data_ptr(), None, q.data_ptr(), m.MTP_DTYPE_F32, 2 * hd, 2 * hd, hd, None, 1e-6, 0.0,
                out.data_ptr(), ws.data_ptr(), size, s.cuda_stream)
        calls.append(lambda args=args: m.lib().mtp_paged_attention(*args))
    torch.cuda.synchronize()
    assert together(calls, 3000) == [0, 0]
    for pool, h, q, out, ln, ws, s in keep:
        assert m.last_error(ws) == m.MTP_OK
        ref, mass, dots = pc.attention(pool, q, None, [16], [1], 0.0)
        assert ((out.double() - ref).abs() <= pc.attention_tol(ref, mass, dots, q.shape[-1], 17, False)).all()


def test_append_of_two_page_sizes():
    import mtp_speculative_decoding_gb300 as m
    calls, keep = [], []
    for page in (256, 128):
        hd, M, s = 512, 200, torch.cuda.Stream()
        pool = pc.Pool(1, 2, page, 1, hd, "e4m3", seed=3)
        h = pool.handle(rope_theta=1e4)
        x = torch.randn(1, M, 1, hd, device="cuda")
        ln = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = m.alloc_workspace(256)
        keep.append((pool, h, x, ln, ws, s))
        args = (C.byref(h), 1, M, ln.data_ptr(), None, x.data_ptr(), x.data_ptr(), m.MTP_DTYPE_F32, M * hd, hd, hd, None, 1e-6,
                ws.data_ptr(), 256, s.cuda_stream)
        calls.append(lambda args=args: m.lib().mtp_kv_append(*args))
    torch.cuda.synchronize()
    assert together(calls, 3000) == [0, 0]
    for _, _, _, _, ws, _ in keep:
        assert m.last_error(ws) == m.MTP_OK
