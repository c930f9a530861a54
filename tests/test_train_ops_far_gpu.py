"""Rows and elements behind 2^32 of a tensor, and parameters off 16-byte
boundaries: layer norm, embedding, their gradients, norm and clipping."""
import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from . import train_ops_reference as R
from .parity import dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _far(rows, n, ld, dtype):
    """rows x n with a row stride that takes the last rows behind element 2^32;
    what lies between is never touched."""
    assert (rows - 1) * ld > 2**32
    return torch.empty((rows - 1) * ld + n, device=dev(), dtype=dtype).as_strided((rows, n), (ld, 1))


def _gen():
    return torch.Generator(device=dev()).manual_seed(3)


def _within(got, ref, bound):
    assert bool(((got.double() - ref).abs() <= bound).all())


# a block a row without the ring, the ring, and single elements
@pytest.mark.parametrize("rows,n,ld", [(70, 320, 2**26), (1300, 320, 2**22), (1300, 321, 2**22 + 1), (70, 20001, 2**26)])
def test_layer_norm_of_rows_behind_four_billion_elements(rows, n, ld):
    g = _gen()
    x, dy = _far(rows, n, ld, BF16), _far(rows, n, ld, BF16)
    x.copy_(torch.randn(rows, n, device=dev(), generator=g))
    dy.copy_(0.1 * torch.randn(rows, n, device=dev(), generator=g))
    w, b = 1 + 0.1 * torch.randn(n, device=dev(), generator=g), torch.randn(n, device=dev(), generator=g)
    mean, rstd = torch.empty(rows, device=dev()), torch.empty(rows, device=dev())
    out = _far(rows, n, ld, BF16)
    B.intlora_layer_norm_batched([B.LayerNormJob(x, w, b, out, mean, rstd)])
    ref, bound = R.layer_norm(x, w, b, 1e-5), R.layer_norm_bounds(x, w, b, 1e-5, BF16)
    for got, r, e in zip((out, mean, rstd), ref, bound):
        _within(got, r, e)
    dw, db = torch.empty(n, device=dev()), torch.empty(n, device=dev())
    jobs = [B.LayerNormBackwardJob(dy, x, w, mean, rstd, out, dw, db)]
    ws = torch.empty(B.intlora_layer_norm_backward_workspace_size(jobs), dtype=torch.uint8, device=dev())
    B.intlora_layer_norm_backward_batched(jobs, ws)
    ref, bound = R.layer_norm_backward(dy, x, w, mean, rstd), R.layer_norm_backward_bounds(dy, x, w, mean, rstd, BF16)
    for got, r, e in zip((out, dw, db), ref, bound):
        _within(got, r, e)


@pytest.mark.parametrize("n", [64, 65])
@pytest.mark.parametrize("tokens", [400, 3000])
def test_embedding_of_words_behind_four_billion_elements(n, tokens):
    g = _gen()
    words, ld = 70, 2**26
    table, y = _far(words, n, ld, BF16), _far(1100, n, 2**22, BF16)
    table.copy_(torch.randn(words, n, device=dev(), generator=g))
    ids = torch.randint(0, words, (tokens,), device=dev(), generator=g)
    ids[-1] = words - 1
    B.intlora_embedding_batched([B.EmbeddingJob(table, ids[:1100], y[:len(ids[:1100])], 2.0)])
    assert torch.equal(y[:len(ids[:1100])].float(), table.float()[ids[:1100]] * 2.0)
    dy = _far(tokens, n, 2**24 if tokens < 1000 else 2**21, BF16)
    whole = torch.randint(-3, 4, (tokens, n), device=dev(), generator=g)
    dy.copy_(whole)
    dtable = table                                # overwritten whole
    jobs = [B.EmbeddingBackwardJob(dy, ids, dtable, 1.0)]
    ws = torch.empty(B.intlora_embedding_backward_workspace_size(jobs), dtype=torch.uint8, device=dev())
    B.intlora_embedding_backward_batched(jobs, ws)
    want = torch.zeros(words, n, device=dev(), dtype=torch.int64).index_add_(0, ids, whole)
    assert torch.equal(dtable.float(), want.to(BF16).float())     # one rounding of an exact sum


def test_norm_and_clipping_of_more_than_four_billion_elements():
    """A norm that is exact: as many ones as 2^32, and 2^18 twos behind them."""
    count = 2**32
    t = torch.ones(count + 2**18, device=dev(), dtype=BF16)
    t[count:] = 2.0
    jobs = [B.GradJob(t)]
    norm = torch.empty(1, device=dev())
    ws = torch.empty(B.intlora_grad_norm_workspace_size(jobs), dtype=torch.uint8, device=dev())
    ref = float(count + 4 * 2**18) ** 0.5
    B.intlora_clip_grad_norm_batched(jobs, ref / 2, norm, ws)
    assert abs(float(norm) - ref) <= R.NORM_RTOL * ref
    # 0.5 and 1 within the factor's error: below half a step of bf16
    assert bool((t[:count:2**16] == 0.5).all()) and bool((t[count - 2**20:count] == 0.5).all())
    assert bool((t[count:] == 1.0).all())


@pytest.mark.parametrize("tokens,n", [(5, 320), (1300, 320), (1300, 4096), (5, 40000)])
@pytest.mark.parametrize("p_dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_parameters_off_sixteen_bytes(tokens, n, p_dtype, shift):
    g = _gen()
    x = torch.randn(tokens, n, device=dev(), generator=g).to(BF16)
    w, b = (torch.randn(n + shift, device=dev(), generator=g).to(p_dtype)[shift:] for _ in range(2))
    y, mean, rstd = torch.empty_like(x), torch.empty(tokens, device=dev()), torch.empty(tokens, device=dev())
    B.intlora_layer_norm_batched([B.LayerNormJob(x, w, b, y, mean, rstd)])
    for got, r, e in zip((y, mean, rstd), R.layer_norm(x, w, b, 1e-5), R.layer_norm_bounds(x, w, b, 1e-5, BF16)):
        _within(got, r, e)
    dx = torch.empty_like(x)
    jobs = [B.LayerNormBackwardJob(y, x, w, mean, rstd, dx)]
    B.intlora_layer_norm_backward_batched(jobs, torch.empty(1, device=dev()))
    _within(dx, R.layer_norm_backward(y, x, w, mean, rstd)[0], R.layer_norm_backward_bounds(y, x, w, mean, rstd, BF16)[0])
