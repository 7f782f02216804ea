"""The paged cache's handle in the binding: which device its tensors live on.
Stand-ins for CUDA tensors, so no GPU is needed; no call reaches the library."""
import gc
import weakref

import pytest
import torch

import mtp_speculative_decoding_gb300 as mtp


class Fake:
    """What the binding asks of a tensor."""

    def __init__(self, shape, dtype=torch.bfloat16, device=0):
        self.like = torch.empty(shape, dtype=dtype, device="meta")
        self.dev = device

    shape = property(lambda s: s.like.shape)
    dtype = property(lambda s: s.like.dtype)
    is_cuda = property(lambda s: s.dev >= 0)
    device = property(lambda s: f"cuda:{s.dev}" if s.dev >= 0 else "cpu")

    def dim(self):
        return self.like.dim()

    def stride(self, *a):
        return self.like.stride(*a)

    def numel(self):
        return self.like.numel()

    def is_contiguous(self):
        return self.like.is_contiguous()

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 1 << 20


class Runtime:
    """The library's place: counts the calls that get through."""

    def __init__(self, device):
        self.calls = []
        self.lib = self
        self.device = lambda: device
        self.raw_stream = lambda d: 0
        self.code = {torch.float32: mtp.MTP_DTYPE_F32, torch.bfloat16: mtp.MTP_DTYPE_BF16}
        self.f32, self.i32 = torch.float32, torch.int32

    def mtp_kv_append(self, *a):
        self.calls.append("append")
        return 0

    def mtp_paged_attention(self, *a):
        self.calls.append("attention")
        return 0


def parts(device, kv=torch.bfloat16):
    d = dict(k=Fake((10, 2, 16, 64), kv, device), v=Fake((10, 2, 16, 64), kv, device),
             page_table=Fake((3, 4), torch.int32, device))
    if kv == torch.float8_e4m3fn:
        d.update(k_scale=Fake((10, 2), torch.float32, device), v_scale=Fake((10, 2), torch.float32, device))
    return d


def both(cache, dev):
    """Both calls with arguments of their own on `dev`."""
    x, ln, ws = Fake((3, 2, 2, 64), device=dev), Fake((3,), torch.int32, dev), Fake((4096,), torch.uint8, dev)
    yield lambda: mtp.kv_append(cache, x, x, ln, ws)
    yield lambda: mtp.paged_attention(cache, x, ln, x, ws)


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_cache_on_another_device_is_refused(monkeypatch, kv):
    """The calls launch on the current device: a cache elsewhere is no argument there."""
    for where, now in ((1, 0), (0, 1), (0, 0), (1, 1)):
        rt = Runtime(now)
        monkeypatch.setattr(mtp, "_runtime", rt)
        cache = mtp.make_kv_cache(**parts(where, kv))
        for call in both(cache, now):
            if where == now:
                call()
            else:
                with pytest.raises(ValueError, match="cuda:%d" % where):
                    call()
        assert rt.calls == (["append", "attention"] if where == now else [])


@pytest.mark.parametrize("other", ["v", "page_table", "k_scale", "v_scale"])
def test_a_cache_on_two_devices_is_refused(other):
    d = parts(0, torch.float8_e4m3fn)
    mtp.make_kv_cache(**d)
    d[other] = parts(1, torch.float8_e4m3fn)[other]
    with pytest.raises(ValueError, match="one device"):
        mtp.make_kv_cache(**d)


def test_a_handle_filled_by_hand_is_taken(monkeypatch):
    """mtp_kv_cache has no device: only make_kv_cache's handles are looked at."""
    rt = Runtime(0)
    monkeypatch.setattr(mtp, "_runtime", rt)
    made = mtp.make_kv_cache(**parts(0))
    by_hand = mtp.KVCache(*[getattr(made, f) for f, _ in mtp.KVCache._fields_])
    for call in both(by_hand, 0):
        call()
    assert rt.calls == ["append", "attention"]


def test_the_handle_keeps_its_tensors():
    """It holds their addresses: a table made in the call's argument list must
    not be freed under it."""
    d = parts(0, torch.float8_e4m3fn)
    refs = [weakref.ref(t) for t in d.values()]
    cache = mtp.make_kv_cache(**d)
    del d
    gc.collect()
    assert all(r() is not None for r in refs)
    del cache
    gc.collect()
    assert all(r() is None for r in refs)
