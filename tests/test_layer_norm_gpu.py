"""Layer norm and its gradients on the GPU against the 64-bit forms, element by
element within bounds derived from fp32 arithmetic (train_ops_reference.py)."""
import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from . import train_ops_reference as R
from .parity import dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GUARD = 77.0


def _strided(tokens, n, dtype, pad, shift):
    """tokens x n inside a larger buffer of GUARD values: row stride n + pad,
    first element `shift` elements behind a 256-byte boundary."""
    buf = torch.full((tokens * (n + pad) + shift + 8,), GUARD, device=dev(), dtype=dtype)
    return buf, buf[shift:shift + tokens * (n + pad)].view(tokens, n + pad)[:, :n]


def _inputs(tokens, n, x_dtype, p_dtype, seed=0, offset=0.3, pad=0, shift=0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=dev(), generator=g)
    _, x = _strided(tokens, n, x_dtype, pad, shift)
    x.copy_(r(tokens, n) * torch.exp(r(tokens, 1)) + offset * r(tokens, 1))
    return x, (1 + 0.2 * r(n)).to(p_dtype), (0.3 * r(n)).to(p_dtype), r


def _forward(x, w, b, y_dtype, eps=1e-5, pad=0, shift=0):
    tokens, n = x.shape
    buf, y = _strided(tokens, n, y_dtype, pad, shift)
    mean, rstd = (torch.full((tokens,), GUARD, device=dev()) for _ in range(2))
    B.intlora_layer_norm_batched([B.LayerNormJob(x, w, b, y, mean, rstd, eps)])
    return buf, y, mean, rstd


def _check_forward(x, w, b, y, mean, rstd, eps=1e-5):
    ry, rm, rr = R.layer_norm(x, w, b, eps)
    by, bm, br = R.layer_norm_bounds(x, w, b, eps, y.dtype)
    for name, got, ref, bound in (("y", y, ry, by), ("mean", mean, rm, bm), ("rstd", rstd, rr, br)):
        over = (got.double() - ref).abs() / bound
        assert float(over.max()) <= 1.0, (name, float(over.max()))


def _backward(dy, x, w, mean, rstd, dx_dtype, pad=0, shift=0, dw=None, db=None, accumulate=False):
    tokens, n = x.shape
    buf, dx = _strided(tokens, n, dx_dtype, pad, shift)
    dw = torch.full((n,), GUARD, device=dev()) if dw is None else dw
    db = torch.full((n,), GUARD, device=dev()) if db is None else db
    jobs = [B.LayerNormBackwardJob(dy, x, w, mean, rstd, dx, dw, db, accumulate)]
    size = B.intlora_layer_norm_backward_workspace_size(jobs)
    ws = torch.full((size + 256,), 0xEE, dtype=torch.uint8, device=dev())
    B.intlora_layer_norm_backward_batched(jobs, ws[:size])
    assert bool((ws[size:] == 0xEE).all())
    return buf, dx, dw, db


def _check_backward(dy, x, w, mean, rstd, dx, dw, db):
    refs = R.layer_norm_backward(dy, x, w, mean, rstd)
    bounds = R.layer_norm_backward_bounds(dy, x, w, mean, rstd, dx.dtype)
    for name, got, ref, bound in zip(("dx", "dweight", "dbias"), (dx, dw, db), refs, bounds):
        err = (got.double() - ref).abs()
        # a sum of terms that are all zero is exactly zero
        over = torch.where(bound > 0, err / bound, err)
        assert float(over.max()) <= 1.0, (name, float(over.max()))


# widths inside a warp (whole chunks and ragged), in a block, at the borders of
# the register forms and behind them
SHAPES = [(1, 1), (3, 1), (1, 8), (5, 7), (2, 9), (17, 33), (40, 64), (9, 255), (9, 256), (9, 257), (7, 320), (33, 640),
          (70, 1001), (5, 1024), (12, 1280), (3, 1288), (6, 2048), (4, 4096), (150, 4096), (149, 4104), (2, 5003),
          (600, 768), (3, 8192), (3, 8200), (2, 16384), (151, 8200), (2, 24576), (2, 24584), (1, 32768), (2, 40001),
          (1, 100000)]


@pytest.mark.parametrize("tokens,n", SHAPES)
def test_shapes(tokens, n):
    x, w, b, r = _inputs(tokens, n, BF16, F32, seed=n)
    _, y, mean, rstd = _forward(x, w, b, BF16)
    _check_forward(x, w, b, y, mean, rstd)
    dy = (0.05 * r(tokens, n))
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, F32)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("tokens,n", [(11, 264), (5, 101), (4, 2056), (3, 9000), (2, 9001), (2, 33000)])
@pytest.mark.parametrize("x_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("y_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("p_dtype", [F32, BF16, F16])
def test_types(tokens, n, x_dtype, y_dtype, p_dtype):
    x, w, b, r = _inputs(tokens, n, x_dtype, p_dtype, seed=7)
    _, y, mean, rstd = _forward(x, w, b, y_dtype)
    _check_forward(x, w, b, y, mean, rstd)
    dy = (0.05 * r(tokens, n)).to(y_dtype)
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, x_dtype)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("n", [8, 100, 320, 1288, 4096, 9000, 40000])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (3, 5), (16, 8)])
def test_strides_and_alignment_leave_what_lies_between(n, pad, shift):
    tokens = 6
    x, w, b, r = _inputs(tokens, n, F16, BF16, seed=n, pad=pad, shift=shift)
    buf, y, mean, rstd = _forward(x, w, b, BF16, pad=pad, shift=shift)
    _check_forward(x, w, b, y, mean, rstd)
    _, dy = _strided(tokens, n, F32, pad, shift)
    dy.copy_(0.05 * r(tokens, n))
    dbuf, dx, dw, db = _backward(dy, x, w, mean, rstd, F16, pad=pad, shift=shift)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)
    for buffer, view in ((buf, y), (dbuf, dx)):
        keep = torch.ones_like(buffer, dtype=torch.bool)
        torch.as_strided(keep, view.shape, view.stride(), view.storage_offset())[:] = False
        assert bool((buffer[keep] == GUARD).all())


@pytest.mark.parametrize("n", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("shift", [0, 1, 3, 6])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_of_which_several_share_sixteen_bytes(n, shift, dtype):
    """Rows shorter than an access, from a base inside one, more of them than
    blocks, so that every place in the ring is used again."""
    tokens = 6000
    x, w, b, r = _inputs(tokens, n, dtype, F32, seed=n, shift=shift)
    buf, y, mean, rstd = _forward(x, w, b, dtype, shift=shift)
    _check_forward(x, w, b, y, mean, rstd)
    _, dy = _strided(tokens, n, dtype, 0, shift)
    dy.copy_(0.05 * r(tokens, n))
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, dtype, shift=shift)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


# more rows than the kernel without a ring takes; half-warp forms of every V
MANY_ROWS = [(1300, 33), (1300, 101), (1300, 255), (1300, 1001), (1300, 5003), (1200, 9001)] + [
    (700, n) for n in (72, 136, 192, 200, 320, 384, 512, 640, 1280, 2048, 16384)]


@pytest.mark.parametrize("tokens,n", MANY_ROWS)
@pytest.mark.parametrize("x_dtype,p_dtype,pad,shift", [(F32, BF16, 0, 0), (BF16, F32, 0, 0), (F16, F16, 8, 0),
                                                       (BF16, F32, 3, 5), (F32, F32, 1, 1)])
def test_many_rows(tokens, n, x_dtype, p_dtype, pad, shift):
    x, w, b, r = _inputs(tokens, n, x_dtype, p_dtype, seed=n, pad=pad, shift=shift)
    _, y, mean, rstd = _forward(x, w, b, x_dtype, pad=pad, shift=shift)
    _check_forward(x, w, b, y, mean, rstd)
    _, dy = _strided(tokens, n, x_dtype, pad, shift)
    dy.copy_(0.05 * r(tokens, n))
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, x_dtype, pad=pad, shift=shift)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("tokens,n", [(5, 264), (1300, 8), (1300, 33), (300, 320), (1300, 1001), (300, 4096), (200, 9000),
                                      (20, 40000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(tokens, n, dtype):
    """y in the place of x, dx in that of dy or of x: the bits of separate tensors."""
    x, w, b, r = _inputs(tokens, n, dtype, F32, seed=n)
    _, y, mean, rstd = _forward(x, w, b, dtype)
    dy = (0.05 * r(tokens, n)).to(dtype)
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, dtype)
    there = x.clone()
    B.intlora_layer_norm_batched([B.LayerNormJob(there, w, b, there)])
    assert torch.equal(there, y)
    for over_x in (False, True):
        xc, dyc = x.clone(), dy.clone()
        dw2, db2 = torch.empty(n, device=dev()), torch.empty(n, device=dev())
        jobs = [B.LayerNormBackwardJob(dyc, xc, w, mean, rstd, xc if over_x else dyc, dw2, db2)]
        ws = torch.empty(B.intlora_layer_norm_backward_workspace_size(jobs), dtype=torch.uint8, device=dev())
        B.intlora_layer_norm_backward_batched(jobs, ws)
        assert torch.equal(xc if over_x else dyc, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("n", [264, 4096])
def test_parts_left_out(n):
    tokens = 200
    x, w, b, r = _inputs(tokens, n, BF16, BF16)
    for wt, bt in ((None, None), (w, None), (None, b)):
        _, y, mean, rstd = _forward(x, wt, bt, F32)
        _check_forward(x, wt, bt, y, mean, rstd)
    y2 = torch.empty_like(y)
    B.intlora_layer_norm_batched([B.LayerNormJob(x, None, b, y2)])
    assert torch.equal(y, y2)
    dy = r(tokens, n).to(BF16)
    _, dx, dw, db = _backward(dy, x, None, mean, rstd, F32)
    _check_backward(dy, x, None, mean, rstd, dx, dw, db)
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    for job in (B.LayerNormBackwardJob(dy, x, None, mean, rstd, dx=dx2),
                B.LayerNormBackwardJob(dy, x, None, mean, rstd, dweight=dw2),
                B.LayerNormBackwardJob(dy, x, None, mean, rstd, dbias=db2)):
        size = B.intlora_layer_norm_backward_workspace_size([job])
        B.intlora_layer_norm_backward_batched([job], torch.empty(max(size, 1), dtype=torch.uint8, device=dev()))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("n", [264, 1001, 4096, 9000])
def test_accumulate_and_same_bits_again(n):
    tokens = 500
    x, w, b, r = _inputs(tokens, n, F32, F32)
    _, y, mean, rstd = _forward(x, w, b, F32)
    dy = r(tokens, n)
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, F32)
    _, dx2, dw2, db2 = _backward(dy, x, w, mean, rstd, F32, dw=torch.ones_like(dw), db=2 * torch.ones_like(db),
                                 accumulate=True)
    assert torch.equal(dx, dx2)
    assert torch.equal(dw2, 1 + dw) and torch.equal(db2, 2 + db)


def test_no_tokens():
    x, w, b, _ = _inputs(1, 64, F32, F32)
    _, y, mean, rstd = _forward(x[:0], w, b, F32)
    dw, db = torch.full((64,), GUARD, device=dev()), torch.full((64,), GUARD, device=dev())
    _backward(x[:0], x[:0], w, mean, rstd, F32, dw=dw, db=db, accumulate=True)
    assert bool((dw == GUARD).all()) and bool((db == GUARD).all())
    _backward(x[:0], x[:0], w, mean, rstd, F32, dw=dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("n", [264, 1001, 4096, 40000])
def test_offsets_constants_and_values_that_are_not_finite(n):
    """A mean far above the spread, a constant row, a row with an infinity and
    one with a NaN: the last two become NaN, and no other row notices."""
    x, w, b, _ = _inputs(9, n, F32, F32)
    x[0] += 3000.0
    x[1] = 5.0
    x[4, n // 2] = float("inf")
    x[6, 0] = float("nan")
    _, y, mean, rstd = _forward(x, w, b, F32)
    bad = [4, 6]
    good = [i for i in range(9) if i not in bad]
    assert bool(torch.isnan(y[bad]).all())
    _check_forward(x[good], w, b, y[good], mean[good], rstd[good])


@pytest.mark.parametrize("n", [3, 20, 33, 40, 264, 520, 1001, 4104, 5003, 9000])
def test_gradient_of_huge_constant_rows(n):
    """xh is zero, although mean rstd is beyond fp32: no column past n may reach
    the sums. rstd is what eps = 1e-5 gives."""
    tokens = 300
    x, w, _, r = _inputs(tokens, n, F32, F32, seed=n)
    x[::2] = 2.0 ** 120
    mean, rstd = x.double().mean(1).float(), torch.full((tokens,), 316.227766, device=dev())
    mean[::2] = 2.0 ** 120
    dy = 0.05 * r(tokens, n)
    _, dx, dw, db = _backward(dy, x, w, mean, rstd, F32)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


def test_jobs_of_one_call_and_streams():
    """Several jobs a call, prebuilt descriptors, and a side stream."""
    sets = [_inputs(t, n, BF16, F32, seed=t) for t, n in ((3, 320), (100, 1280), (1, 4096))]
    want = [_forward(x, w, b, BF16)[1:] for x, w, b, _ in sets]
    got = [tuple(torch.empty_like(t) for t in o) for o in want]
    jobs = B.Descriptors(B.LayerNormJob(x, w, b, *o) for (x, w, b, _), o in zip(sets, got))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.intlora_layer_norm_batched(jobs, stream=side)
    side.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, c))
    dys = [r(*x.shape) for x, _, _, r in sets]
    outs = [_backward(dy, x, w, o[1], o[2], F32)[1:] for dy, (x, w, _, _), o in zip(dys, sets, want)]
    again = [tuple(torch.empty_like(t) for t in o) for o in outs]
    jobs = [B.LayerNormBackwardJob(dy, x, w, o[1], o[2], *a) for dy, (x, w, _, _), o, a in zip(dys, sets, want, again)]
    ws = torch.empty(B.intlora_layer_norm_backward_workspace_size(jobs), dtype=torch.uint8, device=dev())
    with torch.cuda.stream(side):
        B.intlora_layer_norm_backward_batched(jobs, ws)
    side.synchronize()
    for a, c in zip(outs, again):
        assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_gradient_matches_differences_of_the_forward():
    """dx of the kernels against central differences of the 64-bit forward."""
    x, w, b, r = _inputs(2, 24, F32, F32)
    _, y, mean, rstd = _forward(x, w, b, F32)
    dy = r(2, 24)
    _, dx, dw, _ = _backward(dy, x, w, mean, rstd, F32)
    loss = lambda xx, ww: float((R.layer_norm(xx, ww, b, 1e-5)[0] * dy.double()).sum())
    h = 1e-5
    bound = R.layer_norm_backward_bounds(dy, x, w, mean, rstd, F32)
    # the kernels' statistics are fp32: they move dx by up to 40 U of its terms
    slack = 40 * R.U * float(rstd.max() * (dy * w).abs().max() * 24)
    for i in range(24):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[1, i] = h
        diff = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * h)
        assert abs(diff - float(dx[1, i])) < float(bound[0][1, i]) + slack + 1e-6
        e = torch.zeros_like(w, dtype=torch.float64)
        e[i] = h
        diff = (loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * h)
        assert abs(diff - float(dw[i])) < float(bound[1][i]) + slack + 1e-6


# through every form: several rows a warp, half and whole warps, blocks, with and
# without the ring, chunks and single elements, three walks; widths whose 1/n is
# no fp32 number
CONSTANT_ROWS = [(6000, 12), (6000, 40), (1300, 33), (700, 320), (4, 1000), (1300, 1000), (1300, 1001), (1300, 5003),
                 (300, 12000), (200, 22000), (7, 40000), (7, 40001)]


@pytest.mark.parametrize("tokens,n", CONSTANT_ROWS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("eps", [1e-5, 1e-12, 0.0])
def test_constant_rows(tokens, n, dtype, eps):
    """Their mean is the value itself, whatever 1/n rounds to, and their variance
    zero: y is the bias, or with eps = 0 what 0 / 0 gives. The rows between them
    are what they are elsewhere."""
    values = [3.0, 1000.0, 60000.0, -0.1, 7.3e-3] + ([100000.0, 1e-12, -1e-30, 2.3e25] if dtype != F16 else [])
    x, w, b, _ = _inputs(tokens, n, dtype, F32, seed=n)
    rows = torch.arange(tokens, device=dev())
    constant = rows % 3 != 1
    x[constant] = torch.tensor(values, device=dev()).to(dtype)[rows[constant] % len(values)][:, None]
    _, y, mean, rstd = _forward(x, w, b, F32, eps=eps)
    assert torch.equal(mean[constant], x[constant, 0].float())
    if eps > 0:
        assert torch.equal(y[constant], b.expand(int(constant.sum()), n))
        ref = torch.tensor(eps, device=dev()).double() ** -0.5        # eps travels as fp32
        assert bool(((rstd[constant].double() / ref - 1).abs() <= 4 * R.U).all())
    else:
        assert bool(torch.isnan(y[constant]).all()) and bool(torch.isinf(rstd[constant]).all())
    _check_forward(x[~constant], w, b, y[~constant], mean[~constant], rstd[~constant], eps=eps)


@pytest.mark.parametrize("tokens,n", CONSTANT_ROWS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_constant_rows_in_place(tokens, n, dtype):
    """y in the place of x: the bits of separate tensors, with and without parameters."""
    x, w, b, _ = _inputs(tokens, n, dtype, F32, seed=n)
    x[::2] = torch.linspace(-3.0, 70000.0, len(x[::2]), device=dev())[:, None].to(dtype)
    for weight, bias in ((w, b), (None, b), (w, None)):
        _, y, mean, rstd = _forward(x, weight, bias, dtype)
        there = x.clone()
        B.intlora_layer_norm_batched([B.LayerNormJob(there, weight, bias, there)])
        assert torch.equal(there, y)
        assert torch.equal(mean[::2], x[::2, 0].float())
        assert torch.equal(y[::2], (torch.zeros(n, device=dev()) if bias is None else b).to(dtype).expand_as(y[::2]))
