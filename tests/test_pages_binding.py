"""The binding of the operators on pages: views of a model's cache, and what a call writes to."""
import os
import subprocess
import sys

import pytest
import torch

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import pages
from test_pages import gpu, ints, make_cache, make_table

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_expanded_tensors_are_not_written_to():
    x = torch.zeros((4, 3, 2, 8))
    pages._written(x, "x")
    pages._written(x[:1].as_strided((1, 3, 2, 8), (0, 16, 8, 1)), "x")  # one element along the stride of 0
    for bad in (x[:1].expand(4, 3, 2, 8), x[:, :1].expand(4, 3, 2, 8), x[:, :, :1].expand(4, 3, 2, 8)):
        with pytest.raises(ValueError, match="written"):
            pages._written(bad, "x")


@gpu
def test_calls_refuse_expanded_outputs():
    cache = make_cache(torch.int8, 4, 2, 8, 64)
    table, n = make_table(2, 2, 4), ints(9, 9)
    q = torch.randn((2, 1, 4, 64), device="cuda").bfloat16()
    x = torch.empty((2, 1, 2, 64), device="cuda")
    with pytest.raises(ValueError, match="written"):
        cache.attend(table, n, q, out=q[:1].expand(2, 1, 4, 64))
    for k, v in ((x[:1].expand_as(x), x), (x, x[:1].expand_as(x))):
        with pytest.raises(ValueError, match="written"):
            cache.read(table, n - 1, k, v)
    cache.write(table, n, x[:1].expand_as(x), x)  # what is read may be expanded
    assert torch.equal(cache.attend(table, n, q[:1].expand_as(q))[1], cache.attend(table, n, q[:1].repeat(2, 1, 1, 1))[1])


FIRST = """
import sys
import torch
from moe_decode_megakernel_02_gb300 import pages, sampling

def run(what, graph):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    B, Hq, H, D = 20, 8, 2, 128
    L = dict(small=100, pieces=4000, shared=4000)[what]
    cols = L // 64 + 2
    k, v = rand(cols * B, H, 64, D), rand(cols * B, H, 64, D)
    table = torch.arange(cols * B, dtype=torch.int32, device="cuda").view(B, cols)
    if what == "shared":
        table[:, :2] = table[0, :2]
    n, q = torch.full((B,), L, dtype=torch.int32, device="cuda"), rand(B, 1, Hq, D)
    u = torch.full((B,), 0.3, device="cuda")
    p = torch.full((B,), 0.9, device="cuda")
    cache = pages.Pages(k, v)
    def calls():
        cache.write(table, n - 1, q[:, :, :H], q[:, :, H:2 * H])
        out = cache.attend(table, n, q, shared_len=128 if what == "shared" else 0)
        return out, sampling.sample(out.view(B, -1), u, top_p=p)
    if not graph:
        return calls()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = calls()
    gr.replay()
    return out

what = sys.argv[1]
a = run(what, True)
b = run(what, False)
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, b)) and bool(torch.isfinite(a[0].float()).all())
print("same")
"""


@gpu
@pytest.mark.parametrize("what", ["small", "pieces", "shared"])
def test_the_first_calls_of_a_process_may_be_captured(what):
    r = subprocess.run([sys.executable, "-c", FIRST, what], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
