"""Global gradient norm and clipping on the GPU against the 64-bit forms."""
import math

import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from . import train_ops_reference as R
from .parity import dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GUARD = 77.0


def _tensors(counts, dtypes, seed=0, shift=0, scale=1.0):
    """Tensors in one buffer each, between GUARD values."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    out = []
    for k, c in enumerate(counts):
        d = dtypes[k % len(dtypes)]
        buf = torch.full((c + 2 * 16 + shift,), GUARD, device=dev(), dtype=d)
        t = buf[16 + shift:16 + shift + c]
        t.copy_(scale * torch.randn(c, device=dev(), generator=g))
        out.append((buf, t, 16 + shift))
    return out


def _ws(jobs):
    size = B.intlora_grad_norm_workspace_size(jobs)
    return torch.full((max(size, 1),), 0xEE, dtype=torch.uint8, device=dev())


def _norm(ts):
    jobs = [B.GradJob(t) for t in ts]
    norm = torch.full((1,), GUARD, device=dev())
    B.intlora_grad_norm_batched(jobs, norm, _ws(jobs))
    return float(norm)


def _clip(ts, max_norm):
    jobs = [B.GradJob(t) for t in ts]
    norm = torch.full((1,), GUARD, device=dev())
    B.intlora_clip_grad_norm_batched(jobs, max_norm, norm, _ws(jobs))
    return float(norm)


def _check_clipped(before, after, norm, max_norm):
    factor = min(1.0, max_norm / (norm + 1e-6))
    for b, a in zip(before, after):
        want = b.double() * factor
        assert bool(((a.double() - want).abs() <= R.CLIP_RTOL * want.abs() + R.half_step(want, a.dtype)).all())


SETS = [[1], [7], [0, 5, 0], [8191], [8192], [8193], [100_000], [3, 8192 * 5 + 1, 40, 1], [320 * 4] * 256,
        [17] * 1100, [0] * 600 + [33] * 20, [2_000_003, 5]]


@pytest.mark.parametrize("counts", SETS, ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F16, F32, BF16]], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_and_clipping(counts, dtypes, shift):
    made = _tensors(counts, dtypes, seed=len(counts), shift=shift)
    ts = [t for _, t, _ in made]
    before = [t.clone() for t in ts]
    ref = R.grad_norm(ts)
    norm = _norm(ts)
    assert abs(norm - ref) <= R.NORM_RTOL * ref
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    # no clipping: nothing changes
    assert _clip(ts, 2 * ref + 1) == norm
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    # clipping, in both calls the same
    other = [t.clone() for t in ts]
    assert _clip(ts, 0.3 * ref) == norm
    _check_clipped(before, ts, ref, 0.3 * ref)
    B.intlora_grad_clip_batched([B.GradJob(t) for t in other], 0.3 * ref, torch.tensor([norm], device=dev()))
    assert all(torch.equal(t, o) for t, o in zip(ts, other))
    for buf, t, at in made:
        assert bool((buf[:at] == GUARD).all()) and bool((buf[at + t.numel():] == GUARD).all())


@pytest.mark.parametrize("tensors", [63, 64, 65, 255, 256, 257, 511, 512, 513])
def test_tables_of_every_size(tensors):
    counts = [1 + 37 * k % 501 for k in range(tensors)]
    ts = [t for _, t, _ in _tensors(counts, [F32, BF16], seed=tensors)]
    before = [t.clone() for t in ts]
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    assert _norm(ts) == pytest.approx(want, rel=R.NORM_RTOL)
    assert _clip(ts, 1.0) == pytest.approx(want, rel=R.NORM_RTOL)
    _check_clipped(before, ts, want, 1.0)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e18, 1e25, 1e36])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_whose_squares_leave_fp32(scale, dtype):
    ts = [t for _, t, _ in _tensors([20_000, 77], [dtype], scale=scale)]
    ref = R.grad_norm(ts)
    # below fp32's normal numbers storing the norm loses more than half a step
    assert abs(_norm(ts) - ref) <= R.NORM_RTOL * ref + 2.0 ** -149
    before = [t.clone() for t in ts]
    _clip(ts, ref / 2 if ref > 1 else 1e9)
    if ref > 1:
        _check_clipped(before, ts, ref, ref / 2)
    else:
        assert all(torch.equal(t, b) for t, b in zip(ts, before))


def test_one_large_value_among_small_ones():
    t = torch.full((50_000,), 1e-4, device=dev())
    t[31_337] = 3.0
    ref = R.grad_norm([t])
    assert abs(_norm([t]) - ref) <= R.NORM_RTOL * ref


def test_zeros_zero_limit_and_no_tensors():
    z = torch.zeros(10_000, device=dev())
    assert _clip([z], 1.0) == 0.0 and bool((z == 0).all())
    assert _clip([z], 0.0) == 0.0 and bool((z == 0).all())
    t = torch.ones(10_000, device=dev())
    assert abs(_clip([t], 0.0) - 100.0) < 1e-4 and bool((t == 0).all())
    norm = torch.full((1,), GUARD, device=dev())
    B.intlora_grad_norm_batched([], norm)
    assert float(norm) == 0.0
    norm.fill_(GUARD)
    B.intlora_clip_grad_norm_batched([], 1.0, norm)
    assert float(norm) == 0.0
    e = torch.empty(0, device=dev())
    assert _clip([e], 1.0) == 0.0


def test_norms_that_are_not_finite():
    make = lambda: [t for _, t, _ in _tensors([9000, 50], [F32])]
    ts = make()
    ts[1][7] = float("nan")
    assert math.isnan(_clip(ts, 1.0))
    assert all(bool(torch.isnan(t).all()) for t in ts)
    ts = make()
    ts[0][7] = float("inf")
    assert math.isinf(_clip(ts, 1.0))
    assert bool((ts[1] == 0).all()) and math.isnan(float(ts[0][7])) and float(ts[0][8]) == 0.0
    h = torch.full((100,), 60000.0, device=dev(), dtype=F16)     # no infinity: squares are fp32
    assert abs(_norm([h]) - 600_000.0) <= 600_000.0 * R.NORM_RTOL   # 60000 is an fp16 value


def test_same_bits_again_and_descriptors():
    ts = [t for _, t, _ in _tensors([123_457, 9, 70_000], [F32])]
    jobs = B.Descriptors(B.GradJob(t) for t in ts)
    ws = _ws(jobs)
    norms = torch.zeros(3, device=dev())
    for k in range(3):
        B.intlora_grad_norm_batched(jobs, norms[k:k + 1], ws)
    assert norms[0] == norms[1] == norms[2]


def test_ranks_that_hold_parts_of_the_layers():
    """Two sets of tensors, as two ranks hold them: the root of the summed
    squares clips both as one call over all would."""
    parts = [[t for _, t, _ in _tensors([5000, 70], [F32], seed=s)] for s in (1, 2)]
    before = [t.clone() for p in parts for t in p]
    norms = torch.tensor([_norm(p) for p in parts], dtype=torch.float64)
    whole = float((norms ** 2).sum().sqrt())
    ref = R.grad_norm(before)
    assert abs(whole - ref) <= R.NORM_RTOL * ref
    for p in parts:
        B.intlora_grad_clip_batched([B.GradJob(t) for t in p], ref / 3, torch.tensor([whole], device=dev()))
    _check_clipped(before, [t for p in parts for t in p], ref, ref / 3)
