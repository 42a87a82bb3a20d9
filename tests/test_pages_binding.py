"""The binding of the operators on pages: views of a model's cache, and what a call writes to."""
import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import pages
from test_pages import gpu


class _Lib:
    """mk_kv_view of a cache at addresses that nothing follows."""

    @staticmethod
    def mk_kv_view(h, layer, s, t):
        for ref, struct in ((s, mk.PagesStruct(0x1000, 0x2000, None, None, 1024, 512, 64, 0, 0, mk.KV_BF16, 2, 1, 4, 64, 0)),
                            (t, mk.TableStruct(0x3000, 1, 2, 1))):
            ref._obj.__init__(*(getattr(struct, f) for f, _ in struct._fields_))
        return mk.OK


class _Cache:
    h = None


class _Tensor:
    def __init__(self, ptr, device):
        self.ptr, self.device, self.dtype = ptr, device, None

    def data_ptr(self):
        return self.ptr

    def view(self, dtype):
        return self


@pytest.mark.parametrize("current", [0, 1])
def test_a_view_lies_on_the_device_that_holds_the_cache(current, monkeypatch):
    """The cache is on device 1 of 3. Asked for another device, torch gives a copy: what is written there is lost."""
    def as_tensor(data, device=None):
        ptr = data.__cuda_array_interface__["data"][0]
        return _Tensor(ptr if str(device) == "cuda:1" else 0x9000, str(device))

    monkeypatch.setattr(pages, "lib", _Lib)
    monkeypatch.setattr(pages, "Pages", lambda k, v: type("View", (), dict(k=k, v=v))())
    monkeypatch.setattr(torch, "as_tensor", as_tensor)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 3)
    view = pages.of_cache(_Cache(), 0)
    assert [(x.ptr, x.device) for x in (view.k, view.v, view.table)] == [(p, "cuda:1") for p in (0x1000, 0x2000, 0x3000)]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    if current == 0:
        with pytest.raises(RuntimeError):
            pages.of_cache(_Cache(), 0)


@gpu
def test_a_view_is_the_cache_itself():
    from moe_decode_megakernel_02_gb300 import workload
    from synth import configs
    cfg = configs.TINY
    model = workload.load_synthetic(cfg, max_batch=2, max_tokens_per_seq=1, max_ctx=cfg["ctx"] + 8)
    kv = mk.KVCache(model, 2, cfg["ctx"] + 8)
    view, again = kv.pages(0), kv.pages(0)
    assert view.k.data_ptr() == again.k.data_ptr() and view.table.data_ptr() == again.table.data_ptr()
    view.k.fill_(3.0)
    assert bool((again.k == 3).all()) and view.table.tolist() == again.table.tolist()
