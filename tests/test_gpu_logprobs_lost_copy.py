"""mtp_token_logprobs when a copy of logits never arrives: the wait for it ends
after its limit, the row's outputs say that there is no answer, and the other
rows keep theirs.

The kernel's own source is compiled here with its bulk copy replaced by one
that leaves out the copy which covers a given address, so that a wait runs out
(its limit is 20 ms in these calls); nothing is read or written that an
ordinary call does not read or write."""
import ctypes as C
import math
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "common.cuh"
namespace mtp {
__device__ unsigned long long g_left_out;   // an address: the copy that covers it does not start
__device__ __forceinline__ void some_bulk_g2s(void* dst, const void* src, unsigned int bytes, unsigned long long* bar) {
    const unsigned long long at = reinterpret_cast<unsigned long long>(src);
    if (g_left_out >= at && g_left_out < at + bytes) return;
    bulk_g2s(dst, src, bytes, bar);
}
}  // namespace mtp
#define bulk_g2s some_bulk_g2s
#include "logprobs.cu"

extern "C" int leave_out(unsigned long long address) {
    return (int)cudaMemcpyToSymbol(mtp::g_left_out, &address, sizeof address);
}
extern "C" int logprobs(const void* z, int dtype, long long rows, long long V, const int* tokens, int K, float* lp, float* ent, int* ids,
                        float* top, int sms, unsigned long long timeout_ns) {
    mtp::LogprobArgs a;
    a.logits = z; a.rows = rows; a.V = V; a.stride = V; a.tokens = tokens; a.K = K;
    a.logprob = lp; a.entropy = ent; a.top_ids = ids; a.top_logprobs = top;
    a.timeout_ns = timeout_ns;
    return (int)mtp::launch_logprobs(a, dtype, sms, nullptr);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from mtp_speculative_decoding_gb300 import build as b
    d = tmp_path_factory.mktemp("left_out")
    src, so = d / "left_out.cu", d / "libleft_out.so"
    src.write_text(SOURCE)
    cmd = [b._nvcc()] + b._flags() + ["-shared", "-cudart", "shared", str(src), "-o", str(so)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = C.CDLL(str(so))
    P, L64 = C.c_void_p, C.c_longlong
    L.leave_out.argtypes = [C.c_ulonglong]
    L.logprobs.argtypes = [P, C.c_int, L64, L64, P, C.c_int, P, P, P, P, C.c_int, C.c_ulonglong]
    assert os.path.exists(so)
    return L


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [0, 5, 32])
@pytest.mark.parametrize("rows,V", [(3, 200000), (200, 60000), (3, 5000)])      # rows in 16 pieces, in few, in one
def test_a_copy_that_never_arrives(lib, rows, V, K, dtype, code):
    g = torch.Generator(device="cuda").manual_seed(1)
    z = (torch.randn(rows, V, device="cuda", generator=g) * 3).to(dtype)
    tok = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    row = rows // 2

    def call():
        lp, ent = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
        ids = torch.full((rows, max(K, 1)), -7, dtype=torch.int32, device="cuda")
        top = torch.full((rows, max(K, 1)), 7.0, device="cuda")
        assert lib.logprobs(z.data_ptr(), code, rows, V, tok.data_ptr(), K, lp.data_ptr(), ent.data_ptr(),
                            ids.data_ptr() if K else None, top.data_ptr() if K else None, sms, 20_000_000) == 0
        torch.cuda.synchronize()
        return lp, ent, ids, top

    assert lib.leave_out(0) == 0
    whole = call()
    want = torch.log_softmax(z.double(), -1).gather(1, tok.long()[:, None])[:, 0]
    assert ((whole[0].double() - want).abs() <= 1e-4).all()
    others = torch.arange(rows, device="cuda") != row
    for at in (0, V // 7, V // 2, V - 40):
        # an element of a whole 16-byte vector: a row's loose ends are not copied
        assert lib.leave_out(z.data_ptr() + (row * V + at + 8) * z.element_size()) == 0
        got = call()
        assert math.isnan(float(got[0][row])) and math.isnan(float(got[1][row]))
        if K:
            assert (got[2][row] == -1).all() and torch.isnan(got[3][row]).all()
        for a, b in zip(got, whole):
            assert torch.equal(a[others], b[others])
    assert lib.leave_out(0) == 0
    for a, b in zip(call(), whole):
        assert torch.equal(a, b)
