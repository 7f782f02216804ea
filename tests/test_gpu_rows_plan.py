"""The plan of the attention behind shared prefixes at lengths that no cache here
has: the entry point is compiled with the attention and the merge left out, so
that only the kernel that stages the rows and makes the plan runs (it reads no
page), and the plan is read back and compared with whole numbers."""
import ctypes as C
import os
import struct
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "rows_attn_tc.cuh"
namespace mtp {
static cudaError_t no_attention(const RowsTcParams&, cudaStream_t) { return cudaSuccess; }
static cudaError_t no_merge(const RowsTcArgs&, int, cudaStream_t) { return cudaSuccess; }
}  // namespace mtp
#define launch_rows_tc_bf16 no_attention
#define launch_rows_tc_e4m3 no_attention
#define launch_rows_tc_bf16_shared no_attention
#define launch_rows_tc_e4m3_shared no_attention
#define launch_rows_merge no_merge
#include "paged_api.cu"

extern "C" void plan_at(const mtp_kv_cache* c, int B, int M, int n_q_heads, long long* at) {
    const RowsSpace p = rows_space(c, B, M, (int64_t)B * M, n_q_heads, num_sms());
    at[0] = p.head; at[1] = p.worker; at[2] = p.items; at[3] = p.workers; at[4] = p.status;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import mtp_speculative_decoding_gb300 as m
    from mtp_speculative_decoding_gb300 import build as b
    b.build()
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cu", d / "libmtp_plan.so"
    src.write_text(SOURCE)
    objects = [os.path.join(b.BUILD, n + ".o") for n, _, _ in b.UNITS if n != "paged_api"]
    r = subprocess.run([b._nvcc()] + b._flags() + ["-shared", "-cudart", "shared", str(src)] + objects + ["-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = C.CDLL(str(so))
    for name in ("mtp_prefix_workspace_size", "mtp_prefix_attention"):
        f = getattr(L, name)
        f.argtypes, f.restype = getattr(m.lib(), name).argtypes, getattr(m.lib(), name).restype
    L.plan_at.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p]
    L.plan_at.restype = None
    return L


def expected(lens, n, starts, pre, G, hkv):
    """Tiles of the groups' own items (before each of them), units and items in all."""
    items, units, count = [0], 0, 0
    U = 128 * G
    for i, P in enumerate(pre):
        seqs = [(lens[b], n[b]) for b in range(starts[i], starts[i + 1]) if n[b]]
        rows = sum(c for _, c in seqs) * G
        owner = [k for k, (_, c) in enumerate(seqs) for _ in range(c)]            # of a token
        tiles = [(a + c - 1) // 128 - P // 128 + 1 for a, c in seqs]
        rt = -(-rows // 256)
        for x in range(rt):
            r0, r1 = 256 * x, min(rows, 256 * x + 256) - 1
            items.append(items[-1] + sum(tiles[owner[r0 // G]:owner[r1 // G] + 1]))
        units += (rt * -(-P // 128) + items[-1] - items[-1 - rt]) * U * hkv
        count += hkv * (rt * (2 if P else 1))
    return items, units, count


@pytest.mark.parametrize("B,M,G,hkv,groups", [(127, 64, 16, 1, 1), (120, 63, 16, 2, 3), (100, 33, 7, 1, 2), (5, 4, 4, 1, 1)])
def test_tiles_are_counted_beyond_31_bits(lib, B, M, G, hkv, groups):
    import mtp_speculative_decoding_gb300 as m
    hd, page = 64, 256
    max_pages = 0x7FFFFF00 // page
    cap = max_pages * page
    kv = torch.zeros((1, hkv, page, hd), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")               # (the plan reads no page)
    h = m.make_kv_cache(kv, kv, table, rope_theta=1e4)
    h.max_pages = max_pages
    g = torch.Generator().manual_seed(1)
    starts = [B * i // groups for i in range(groups + 1)]
    pre = torch.randint(0, 100000, (groups,), generator=g).tolist()
    n = torch.randint(1, M + 1, (B,), generator=g).tolist()
    n[0], n[-1] = M, M
    if B > 100:
        n = [M] * B
    lens = [cap - c - int(x) for c, x in zip(n, torch.randint(0, 1000, (B,), generator=g))]
    q = torch.zeros((B, M, hkv * G, hd), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((1, 1, 1, hd), dtype=torch.bfloat16, device="cuda")       # (nor does it write a result)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")           # noqa: E731
    dev = i32(lens), i32(n), i32(starts), i32(pre)
    size = lib.mtp_prefix_workspace_size(C.byref(h), B, M, hkv * G)
    assert size > 0
    ws = m.alloc_workspace(size)
    rc = lib.mtp_prefix_attention(C.byref(h), B, M, hkv * G, dev[0].data_ptr(), dev[1].data_ptr(), groups, dev[2].data_ptr(), dev[3].data_ptr(),
                                  q.data_ptr(), m.MTP_DTYPE_BF16, q.stride(0), q.stride(1), q.stride(2), None, 1e-6, 0.0, out.data_ptr(),
                                  ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == m.MTP_OK
    torch.cuda.synchronize()
    at = (C.c_longlong * 5)()
    lib.plan_at(C.byref(h), B, M, hkv * G, at)
    mem = ws.cpu().numpy().tobytes()
    items, units, count = expected(lens, n, starts, pre, G, hkv)
    assert list(struct.unpack_from(f"{len(items)}q", mem, at[2])) == items
    if B > 100:
        assert items[-1] > 2 ** 32
    T, opened, workers = struct.unpack_from("qii", mem, at[0])
    assert workers == at[3] and T == units + count * opened * 128 * G
    assert struct.unpack_from("i", mem, at[4] + 4 * workers)[0] == m.MTP_OK
    end = 0
    for w in range(workers):      # even shares of the line, each with an item that begins at its start or in front of it
        xs, xe, begin, blk = struct.unpack_from("qqqi", mem, at[1] + 96 * w)
        assert xs == end and xe - xs in (T // workers, T // workers + 1) and 0 <= begin <= xs
        assert 0 <= blk < 2 * groups
        end = xe
    assert end == T
