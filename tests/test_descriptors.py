"""Prebuilt descriptor lists hold addresses: the tensors behind them must live as
long."""
import gc
import weakref

import torch

from quantized_lora_merge_b200 import binding as B


def test_tensors_live_as_long_as_the_descriptors(monkeypatch):
    monkeypatch.setattr(B, "_one_device", lambda *t: None)         # no GPU here
    x, w, b, y = torch.randn(4, 8), torch.randn(8), torch.randn(8), torch.empty(4, 8)
    refs = [weakref.ref(t) for t in (x, w, b, y)]
    want = [t.data_ptr() for t in (x, w, b, y)]
    jobs = B.Descriptors(B.LayerNormJob(*t) for t in [(x, w, b, y)])
    del x, w, b, y
    gc.collect()
    assert all(r() is not None for r in refs)
    c = jobs.arr[0]
    assert [c.x, c.weight, c.bias, c.y] == want
    del jobs, c
    gc.collect()
    assert all(r() is None for r in refs)
