"""Layer norm, embedding, gradient norm and clipping without a GPU: the C ABI
refuses bad arguments on the host (no call here reaches a launch), the binding
refuses tensors it cannot describe, and the 64-bit reference that the GPU tests
use is itself checked against differences."""
import ctypes

import pytest
import torch

from quantized_lora_merge_b200 import binding as B
from quantized_lora_merge_b200.build import build

from . import train_ops_reference as R

FAKE = 0x100000  # 256-byte-aligned dummy address; never dereferenced by validation


@pytest.fixture(scope="module")
def lib():
    build()
    return B.lib()


def _job(struct, base, **kw):
    f = dict(base)
    f.update(kw)
    return (struct * 1)(struct(**f))


LN = dict(x=FAKE, weight=FAKE, bias=FAKE, y=FAKE, mean=FAKE, rstd=FAKE, tokens=4, n=16, ld_x=16, ld_y=16, x_type=1,
          param_type=0, y_type=1, eps=1e-5)
LNB = dict(dy=FAKE, x=FAKE, weight=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dweight=FAKE, dbias=FAKE, tokens=4, n=16,
           ld_dy=16, ld_x=16, ld_dx=16, dy_type=0, x_type=1, param_type=0, dx_type=0, accumulate=0)
EMB = dict(table=FAKE, ids=FAKE, y=FAKE, invalid=FAKE, vocab=10, n=16, tokens=4, ld_table=16, ld_y=16, table_type=1,
           y_type=1, id_bytes=8, scale=1.0)
EMBB = dict(dy=FAKE, ids=FAKE, dtable=FAKE, invalid=FAKE, vocab=10, n=16, tokens=4, padding_id=-1, ld_dy=16,
            ld_dtable=16, dy_type=1, dtable_type=0, id_bytes=8, accumulate=0, scale=1.0)

BAD_SIZES = [("n", 0, "n >= 1"), ("n", -8, "n >= 1"), ("tokens", -1, "tokens >= 0"), ("tokens", 2**31, "2^31"),
             ("n", 2**31, "2^31")]


@pytest.mark.parametrize("field,value,needle", BAD_SIZES + [
    ("x", None, "x and y"), ("y", None, "x and y"), ("x_type", 3, "types"), ("param_type", -1, "types"),
    ("y_type", 7, "types"), ("eps", -1.0, "eps"), ("eps", float("nan"), "eps"), ("eps", float("inf"), "eps"),
    ("ld_x", 15, "ld_x"), ("ld_y", 0, "ld_y"), ("ld_x", 2**40, "2^40"), ("x", FAKE + 1, "aligned"),
    ("weight", FAKE + 2, "aligned"), ("mean", FAKE + 2, "aligned")])
def test_layer_norm_rejects(lib, field, value, needle):
    jobs = _job(B.intlora_layer_norm_job, LN, **{field: value})
    assert lib.intlora_layer_norm_batched(jobs, 1, None) == 1
    assert needle in lib.intlora_last_error().decode()


@pytest.mark.parametrize("field,value,needle", BAD_SIZES + [
    ("dy", None, "required"), ("x", None, "required"), ("mean", None, "required"), ("rstd", None, "required"),
    ("dx_type", 3, "types"), ("ld_dx", 8, "ld_dx"), ("ld_dy", 8, "ld_dy"), ("dy", FAKE + 2, "aligned"),
    ("dweight", FAKE + 1, "aligned")])
def test_layer_norm_backward_rejects(lib, field, value, needle):
    jobs = _job(B.intlora_layer_norm_backward_job, LNB, **{field: value})
    assert lib.intlora_layer_norm_backward_batched(jobs, 1, FAKE, 1 << 30, None) == 1
    assert needle in lib.intlora_last_error().decode()


def test_layer_norm_backward_workspace_checked(lib):
    jobs = _job(B.intlora_layer_norm_backward_job, LNB)
    need = lib.intlora_layer_norm_backward_workspace_size(jobs, 1)
    assert need > 0 and need % 256 == 0
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert lib.intlora_layer_norm_backward_batched(jobs, 1, ws, size, None) == 3
        assert str(need) in lib.intlora_last_error().decode()
    only_dx = _job(B.intlora_layer_norm_backward_job, LNB, dweight=None, dbias=None)
    assert lib.intlora_layer_norm_backward_workspace_size(only_dx, 1) == 0
    two = (B.intlora_layer_norm_backward_job * 2)(jobs[0], jobs[0])
    assert lib.intlora_layer_norm_backward_workspace_size(two, 2) == 2 * need


@pytest.mark.parametrize("field,value,needle", BAD_SIZES + [
    ("table", None, "required"), ("ids", None, "required"), ("y", None, "required"), ("vocab", 0, "vocab"),
    ("vocab", 2**31, "vocab"), ("id_bytes", 2, "id_bytes"), ("table_type", 5, "types"), ("ld_table", 8, "ld_table"),
    ("ld_y", 8, "ld_y"), ("ids", FAKE + 4, "aligned"), ("invalid", FAKE + 2, "aligned"),
    ("table", FAKE + 1, "aligned")])
def test_embedding_rejects(lib, field, value, needle):
    jobs = _job(B.intlora_embedding_job, EMB, **{field: value})
    assert lib.intlora_embedding_batched(jobs, 1, None) == 1
    assert needle in lib.intlora_last_error().decode()


@pytest.mark.parametrize("field,value,needle", BAD_SIZES + [
    ("dtable", None, "dtable"), ("ids", None, "required"), ("dy", None, "required"), ("vocab", -1, "vocab"),
    ("id_bytes", 1, "id_bytes"), ("dtable_type", 4, "types"), ("ld_dtable", 8, "ld_dtable"), ("ld_dy", 8, "ld_dy"),
    ("dtable", FAKE + 2, "aligned")])
def test_embedding_backward_rejects(lib, field, value, needle):
    jobs = _job(B.intlora_embedding_backward_job, EMBB, **{field: value})
    assert lib.intlora_embedding_backward_batched(jobs, 1, FAKE, 1 << 30, None) == 1
    assert needle in lib.intlora_last_error().decode()


@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_embedding_rejects_a_scale_that_makes_missing_rows_nan(lib, scale):
    jobs = _job(B.intlora_embedding_job, EMB, scale=scale)
    assert lib.intlora_embedding_batched(jobs, 1, None) == 1
    assert "scale" in lib.intlora_last_error().decode()
    jobs = _job(B.intlora_embedding_backward_job, EMBB, scale=scale)
    assert lib.intlora_embedding_backward_batched(jobs, 1, FAKE, 1 << 30, None) == 1
    assert "scale" in lib.intlora_last_error().decode()


def test_embedding_backward_workspace_checked(lib):
    jobs = _job(B.intlora_embedding_backward_job, EMBB, tokens=1000)
    need = lib.intlora_embedding_backward_workspace_size(jobs, 1)
    assert need >= 1000 * 16 and need % 256 == 0
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 128, need)):
        assert lib.intlora_embedding_backward_batched(jobs, 1, ws, size, None) == 3


def _grads(*items):
    return (B.intlora_grad_job * len(items))(*[B.intlora_grad_job(*i) for i in items])


@pytest.mark.parametrize("items,needle", [
    ([(FAKE, -1, 0)], "count"), ([(FAKE, 4, 3)], "type"), ([(None, 4, 0)], "NULL"), ([(FAKE + 2, 4, 0)], "aligned"),
    ([(FAKE + 1, 4, 1)], "aligned"), ([(FAKE, 2**40, 0), (FAKE, 1, 0)], "2^40")])
def test_gradients_rejected(lib, items, needle):
    jobs = _grads(*items)
    for call in (lambda: lib.intlora_grad_norm_batched(jobs, len(items), FAKE, FAKE, 1 << 20, None),
                 lambda: lib.intlora_grad_clip_batched(jobs, len(items), 1.0, FAKE, None),
                 lambda: lib.intlora_clip_grad_norm_batched(jobs, len(items), 1.0, FAKE, FAKE, 1 << 20, None)):
        assert call() == 1
        assert needle in lib.intlora_last_error().decode()


def test_clipping_rejects_overlaps_and_bad_norms(lib):
    # the same tensor twice, a tensor inside another, an overlap out of order
    for items in ([(FAKE, 4, 0), (FAKE, 4, 0)], [(FAKE, 100, 0), (FAKE + 64, 2, 1)],
                  [(FAKE + 4096, 8, 0), (FAKE, 1025, 0)]):
        jobs = _grads(*items)
        assert lib.intlora_clip_grad_norm_batched(jobs, 2, 1.0, FAKE, FAKE, 1 << 20, None) == 1
        assert lib.intlora_last_error().decode() == "gradient jobs 0 and 1 overlap"
        assert lib.intlora_grad_clip_batched(jobs, 2, 1.0, FAKE, None) == 1
    jobs = _grads((FAKE, 4, 0))
    for bad in (-1.0, float("nan"), float("inf")):
        assert lib.intlora_clip_grad_norm_batched(jobs, 1, bad, FAKE, FAKE, 1 << 20, None) == 1
        assert "max_norm" in lib.intlora_last_error().decode()
    assert lib.intlora_clip_grad_norm_batched(jobs, 1, 1.0, None, FAKE, 1 << 20, None) == 1
    assert lib.intlora_grad_clip_batched(jobs, 1, 1.0, FAKE + 2, None) == 1
    assert lib.intlora_grad_norm_batched(jobs, 1, FAKE, None, 0, None) == 3
    assert lib.intlora_clip_grad_norm_batched(jobs, 1, 1.0, FAKE, FAKE, 0, None) == 3


def test_empty_calls_are_no_ops(lib):
    assert lib.intlora_layer_norm_batched(None, 0, None) == 0
    assert lib.intlora_layer_norm_batched(_job(B.intlora_layer_norm_job, LN, tokens=0, x=None, y=None), 1, None) == 0
    assert lib.intlora_layer_norm_backward_batched(None, 0, None, 0, None) == 0
    assert lib.intlora_embedding_batched(_job(B.intlora_embedding_job, EMB, tokens=0), 1, None) == 0
    assert lib.intlora_embedding_backward_batched(None, 0, None, 0, None) == 0
    none = _job(B.intlora_embedding_backward_job, EMBB, tokens=0, accumulate=1, dy=None, ids=None)
    assert lib.intlora_embedding_backward_workspace_size(none, 1) == 0
    assert lib.intlora_embedding_backward_batched(none, 1, None, 0, None) == 0
    assert lib.intlora_grad_clip_batched(None, 0, 1.0, FAKE, None) == 0
    for call in (lib.intlora_layer_norm_batched,):
        assert call(None, 1, None) == 1 and call(None, -1, None) == 1


def test_binding_refuses_what_it_cannot_describe():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        B.LayerNormJob(x, None, None, x).to_c()
    with pytest.raises(ValueError, match="CUDA"):
        B.GradJob(x).to_c()
    with pytest.raises(ValueError, match="CUDA"):
        B.EmbeddingJob(x, torch.zeros(3, dtype=torch.int64), x).to_c()
    with pytest.raises(ValueError, match="contiguous"):
        B._matrix("x", torch.zeros(16, 4).t())
    with pytest.raises(ValueError, match="2-D"):
        B._matrix("x", torch.zeros(2, 3, 4))
    with pytest.raises(ValueError, match="4 x 16"):
        B._matrix("y", torch.zeros(4, 15), 4, 16)
    with pytest.raises(TypeError, match="fp32, bf16 or fp16"):
        B._elem_type("x", torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="vector of 8"):
        B._vector("weight", torch.zeros(7), 8)
    with pytest.raises(TypeError, match="int32 or int64"):
        B._ids(torch.zeros(2, dtype=torch.int16))
    with pytest.raises(TypeError, match="norm"):
        B._norm_scalar(torch.zeros(2))
    assert B._matrix("x", torch.zeros(4, 20)[:, 2:18]) == 20
    assert B._matrix("x", torch.zeros(1, 16).expand(1, 16)) == 16


def test_binding_refuses_workspaces_and_norms_elsewhere(monkeypatch):
    class On:
        def __init__(self, device, contiguous=True):
            self.device, self.contiguous = torch.device(device), contiguous

        def get_device(self):
            return -1 if self.device.index is None else self.device.index

        def is_contiguous(self):
            return self.contiguous

    class Job:
        def device(self):
            return torch.device("cuda:0")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    B._here([Job()], On("cuda:0"), None)
    B._here([], None)
    for jobs, other, needle in (([Job()], On("cpu"), "CUDA"), ([Job()], On("cuda:1"), "on cuda:1, other tensors on cuda:0"),
                                ([], On("cuda:1"), "cuda:1"), ([Job()], On("cuda:0", False), "contiguous")):
        with pytest.raises(ValueError, match=needle):
            B._here(jobs, other)
    with pytest.raises(ValueError, match="CUDA"):
        B.intlora_layer_norm_backward_batched([], torch.empty(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        B.intlora_embedding_backward_batched([], torch.empty(256, dtype=torch.uint8))
    with pytest.raises((TypeError, ValueError), match="CUDA"):
        B.intlora_clip_grad_norm_batched([], 1.0, torch.zeros(1), torch.empty(256, dtype=torch.uint8))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        B._here([Job()])


def test_header_accepts_the_descriptors_in_c(tmp_path):
    import shutil
    import subprocess
    from pathlib import Path
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src = tmp_path / "use.c"
    src.write_text(r'''
#include "intlora.h"
int use(void* p) {
  intlora_layer_norm_job a = {p, p, p, p, 0, 0, 1, 8, 8, 8, INTLORA_TYPE_BF16, INTLORA_TYPE_F32, INTLORA_TYPE_F16, 1e-5f};
  intlora_layer_norm_backward_job b = {p, p, p, p, p, p, p, p, 1, 8, 8, 8, 8, 0, 1, 0, 0, 1};
  intlora_embedding_job c = {p, p, p, p, 10, 8, 1, 8, 8, 0, 1, 8, 2.0f};
  intlora_embedding_backward_job d = {p, p, p, p, 10, 8, 1, -1, 8, 8, 0, 0, 4, 1, 2.0f};
  intlora_grad_job e = {p, 8, INTLORA_TYPE_F32};
  return (int)(a.eps + b.accumulate + c.scale + d.scale + e.count);
}
''')
    inc = Path(__file__).resolve().parents[1] / "include"
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-c", str(src), "-I", str(inc),
                          "-o", str(tmp_path / "use.o")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


# ---------------------------------------------------------------------------
# the reference's gradients against central differences in 64 bits
# ---------------------------------------------------------------------------
def test_reference_layer_norm_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 7, generator=g, dtype=torch.float64)
    w = torch.randn(7, generator=g, dtype=torch.float64)
    b = torch.randn(7, generator=g, dtype=torch.float64)
    dy = torch.randn(3, 7, generator=g, dtype=torch.float64)
    _, mean, rstd = R.layer_norm(x, w, b, 1e-5)
    grads = R.layer_norm_backward(dy, x, w, mean, rstd)
    h = 1e-6
    for t, got in zip((x, w, b), grads):
        flat = t.view(-1)
        for i in range(flat.numel()):
            old = flat[i].item()
            losses = []
            for v in (old + h, old - h):
                flat[i] = v
                losses.append(float((R.layer_norm(x, w, b, 1e-5)[0] * dy).sum()))
            flat[i] = old
            # the truncation is of order h^2 and the cancellation of order 2^-53 / h
            assert abs((losses[0] - losses[1]) / (2 * h) - float(got.view(-1)[i])) < 1e-7


def test_reference_embedding_gradient_matches_differences():
    g = torch.Generator().manual_seed(4)
    table = torch.randn(5, 3, generator=g, dtype=torch.float64)
    ids = torch.tensor([4, 0, 4, 2, 4, -1, 9])
    dy = torch.randn(7, 3, generator=g, dtype=torch.float64)
    got, _, count = R.embedding_backward(dy, ids, 5, 2.5)
    assert count.tolist() == [1, 0, 1, 0, 3]
    for i in range(15):
        e = torch.zeros(15, dtype=torch.float64)
        e[i] = 1.0
        # the lookup is linear in the table: its difference is exact
        diff = ((R.embedding(e.view(5, 3), ids, 2.5)) * dy).sum()
        assert abs(float(diff) - float(got.view(-1)[i])) < 1e-13
