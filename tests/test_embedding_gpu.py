"""Embedding lookup and its gradient by sorted tokens on the GPU against the
64-bit forms, within bounds derived from fp32 arithmetic."""
import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from . import train_ops_reference as R
from .parity import dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GUARD = 77.0


def _gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def _rows(rows, n, dtype, gen, pad=0, shift=0):
    buf = torch.full((rows * (n + pad) + shift + 8,), GUARD, device=dev(), dtype=dtype)
    view = buf[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]
    if gen is not None:
        view.copy_(torch.randn(rows, n, device=dev(), generator=gen))
    return buf, view


def _only_view_written(buf, view):
    keep = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(keep, view.shape, view.stride(), view.storage_offset())[:] = False
    return bool((buf[keep] == GUARD).all())


def _lookup(table, ids, scale, y_dtype, pad=0, shift=0):
    buf, y = _rows(ids.numel(), table.shape[1], y_dtype, None, pad, shift)
    bad = torch.zeros(1, dtype=torch.int32, device=dev())
    B.intlora_embedding_batched([B.EmbeddingJob(table, ids, y, scale, bad)])
    assert _only_view_written(buf, y)
    return y, int(bad)


def _check_lookup(table, ids, scale, y):
    ref = R.embedding(table, ids, scale)
    bound = R.U * ref.abs() + R.half_step(ref, y.dtype)
    assert bool(((y.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("tokens,vocab,n", [(1, 1, 1), (1, 50, 4096), (8, 1000, 4096), (7, 10, 3), (300, 77, 40),
                                            (5000, 100, 64), (1000, 2000, 768), (33, 9, 8200), (3000, 50, 1001)])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
def test_lookup_shapes(tokens, vocab, n, id_dtype):
    g = _gen(n)
    _, table = _rows(vocab, n, BF16, g)
    ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g).to(id_dtype)
    y, bad = _lookup(table, ids, 3.5, BF16)
    assert bad == 0
    _check_lookup(table, ids, 3.5, y)


@pytest.mark.parametrize("t_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("y_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 3)])
def test_lookup_types_and_strides(t_dtype, y_dtype, pad, shift):
    g = _gen(5)
    _, table = _rows(60, 136, t_dtype, g, pad, shift)
    ids = torch.randint(0, 60, (50,), device=dev(), generator=g)
    y, _ = _lookup(table, ids, 0.37, y_dtype, pad, shift)
    _check_lookup(table, ids, 0.37, y)


@pytest.mark.parametrize("n", [5, 64, 4096])
def test_lookup_of_ids_outside_the_table(n):
    g = _gen(6)
    _, table = _rows(20, n, F32, g)
    ids = torch.tensor([0, -1, 19, 20, 2**40, -2**62, 3, 2**31], device=dev())
    y, bad = _lookup(table, ids, 2.0, F32)
    assert bad == 5
    _check_lookup(table, ids, 2.0, y)
    y, bad = _lookup(table, torch.tensor([5, -7, 2**31 - 1], device=dev(), dtype=torch.int32), 2.0, F32)
    assert bad == 2 and bool((y[1:] == 0).all())


def _backward(dy, ids, vocab, scale=1.0, dtype=F32, padding_id=-1, old=None, pad=0, shift=0):
    buf, dtable = _rows(vocab, dy.shape[1], dtype, None, pad, shift)
    if old is not None:
        dtable.copy_(old)
    bad = torch.zeros(1, dtype=torch.int32, device=dev())
    jobs = [B.EmbeddingBackwardJob(dy, ids, dtable, scale, padding_id, old is not None, bad)]
    size = B.intlora_embedding_backward_workspace_size(jobs)
    ws = torch.full((size + 256,), 0xEE, dtype=torch.uint8, device=dev())
    B.intlora_embedding_backward_batched(jobs, ws[:size])
    assert bool((ws[size:] == 0xEE).all())
    assert _only_view_written(buf, dtable)
    return dtable, int(bad)


def _check_backward(dy, ids, vocab, dtable, scale=1.0, padding_id=-1, old=None):
    out, mag, count = R.embedding_backward(dy, ids, vocab, scale, padding_id, old)
    err = (dtable.double() - out).abs()
    bound = R.embedding_backward_bound(out, mag, count, dtable.dtype)
    touched = count > 0
    assert bool((err[touched] <= bound[touched]).all()), float((err / bound)[touched].max())
    if old is None:
        assert bool((dtable[~touched] == 0).all())
    else:
        assert torch.equal(dtable[~touched].view(-1), old.to(dtable.dtype)[~touched].view(-1))


# lengths around the chunks of 32, the runs of 256, and the joined runs of 16384
LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 511, 512, 513, 1000, 4097, 16383, 16384, 16385, 40000]


@pytest.mark.parametrize("tokens", LENGTHS)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("law", ["uniform", "few", "one word", "distinct"])
def test_gradient_lengths_and_laws(tokens, accumulate, law):
    vocab, n = (50000, 8) if law in ("uniform", "distinct") else (40, 24)
    g = _gen(tokens)
    _, dy = _rows(tokens, n, F32, g)
    if law == "distinct":
        ids = torch.randperm(vocab, device=dev(), generator=g)[:tokens]
    elif law == "one word":
        ids = torch.full((tokens,), 17, device=dev())
    else:
        ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g)
    old = _rows(vocab, n, F32, g)[1] if accumulate else None
    dtable, bad = _backward(dy, ids, vocab, 2.5, old=old)
    assert bad == 0
    _check_backward(dy, ids, vocab, dtable, 2.5, old=old)


@pytest.mark.parametrize("tokens,n,vocab", [(300, 1, 20), (300, 3, 20), (77, 768, 500), (600, 4096, 30), (500, 4100, 9),
                                            (200, 8200, 3), (130, 1001, 1), (40, 20000, 2)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_widths(tokens, n, vocab, accumulate):
    g = _gen(n)
    _, dy = _rows(tokens, n, BF16, g)
    ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g).int()
    old = _rows(vocab, n, F32, g)[1] if accumulate else None
    dtable, _ = _backward(dy, ids, vocab, 0.5, old=old)
    _check_backward(dy, ids, vocab, dtable, 0.5, old=old)


@pytest.mark.parametrize("tokens,n,vocab", [(700, 4100, 9), (600, 1001, 5), (600, 8200, 3), (900, 1, 2), (513, 20008, 200),
                                            (1500, 129, 70)])
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_widths_of_sorted_texts(tokens, n, vocab, dtype, accumulate):
    g = _gen(n)
    _, dy = _rows(tokens, n, dtype, g)
    ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g)
    old = _rows(vocab, n, F32, g)[1] if accumulate else None
    dtable, _ = _backward(dy, ids, vocab, 0.5, old=old)
    _check_backward(dy, ids, vocab, dtable, 0.5, old=old)


@pytest.mark.parametrize("counts", [[1] * 120 + [600, 1, 16, 17, 9, 8, 300], [127, 1, 700, 31, 33, 64, 65, 7],
                                    [96, 31, 2, 513, 128, 128, 129, 40], [2000], [5, 640, 3, 544, 4]])
@pytest.mark.parametrize("n", [24, 264, 301, 2056])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_words_across_windows(counts, n, accumulate):
    """Words of every frequency that begin and end at, before and behind the
    borders of 32 and of 128 sorted positions."""
    g = _gen(n)
    ids = torch.repeat_interleave(torch.arange(len(counts), device=dev()), torch.tensor(counts, device=dev()))
    ids = ids[torch.randperm(ids.numel(), device=dev(), generator=g)]
    vocab = len(counts) + 3
    _, dy = _rows(ids.numel(), n, BF16, g)
    old = _rows(vocab, n, F32, g)[1] if accumulate else None
    dtable, _ = _backward(dy, ids, vocab, 1.0, old=old)
    _check_backward(dy, ids, vocab, dtable, 1.0, old=old)


@pytest.mark.parametrize("dy_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (16, 8), (1, 3)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_types_and_strides(dy_dtype, dtype, pad, shift, accumulate):
    g = _gen(8)
    _, dy = _rows(700, 136, dy_dtype, g, pad, shift)
    ids = torch.randint(0, 30, (700,), device=dev(), generator=g)
    old = _rows(30, 136, F32, g)[1].to(dtype) if accumulate else None
    dtable, _ = _backward(dy, ids, 30, 1.5, dtype, old=old, pad=pad, shift=shift)
    _check_backward(dy, ids, 30, dtable, 1.5, old=old)


@pytest.mark.parametrize("tokens", [20, 500, 20000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_with_padding_and_ids_outside_the_table(tokens, accumulate):
    """The padding id's row gets nothing (zeros, or its old values), ids outside
    are counted; values that are not finite in their rows reach nobody."""
    vocab, n = 30, 40
    g = _gen(tokens)
    _, dy = _rows(tokens, n, F32, g)
    ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g)
    ids[1::4] = 5
    ids[2::9] = -3
    ids[3::9] = vocab
    ids[4] = 2**40
    away = (ids == 5) | (ids < 0) | (ids >= vocab)
    dy[away] = float("nan")
    old = _rows(vocab, n, F32, g)[1] if accumulate else None
    dtable, bad = _backward(dy, ids, vocab, padding_id=5, old=old)
    assert bad == int(((ids < 0) | (ids >= vocab)).sum())
    assert bool(torch.isfinite(dtable).all())
    _check_backward(torch.nan_to_num(dy), ids, vocab, dtable, padding_id=5, old=old)


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_nothing_but_padding_and_of_no_tokens(accumulate):
    old = _rows(12, 16, F32, _gen(1))[1] if accumulate else None
    want = old if accumulate else torch.zeros(12, 16, device=dev())
    for tokens in (0, 1, 400):
        dy = torch.full((tokens, 16), float("nan"), device=dev())
        dtable, _ = _backward(dy, torch.full((tokens,), 3, device=dev()), 12, padding_id=3, old=old)
        assert torch.equal(dtable, want)


def test_gradient_same_bits_again_and_jobs_of_one_call():
    g = _gen(2)
    jobs, outs, want = [], [], []
    for tokens, n, vocab in ((5000, 136, 40), (100, 768, 300), (20000, 24, 7)):
        _, dy = _rows(tokens, n, BF16, g)
        ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=g)
        want.append(_backward(dy, ids, vocab, 3.0)[0])
        assert torch.equal(want[-1], _backward(dy, ids, vocab, 3.0)[0])
        outs.append(torch.empty(vocab, n, device=dev()))
        jobs.append(B.EmbeddingBackwardJob(dy, ids, outs[-1], 3.0))
    jobs = B.Descriptors(jobs)
    ws = torch.empty(B.intlora_embedding_backward_workspace_size(jobs), dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.intlora_embedding_backward_batched(jobs, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_gradient_matches_differences_of_the_lookup():
    """The lookup is linear: dtable[v, c] is the loss of the unit table."""
    g = _gen(3)
    ids = torch.tensor([4, 0, 4, 2, 4, 3, 3, -1], device=dev())
    _, dy = _rows(8, 8, F32, g)
    dtable, _ = _backward(dy, ids, 5, 1.5)
    for v in range(5):
        for c in range(8):
            unit = torch.zeros(5, 8, device=dev())
            unit[v, c] = 1.0
            y, _ = _lookup(unit, ids, 1.5, F32)
            diff = float((y.double() * dy.double()).sum())
            assert abs(diff - float(dtable[v, c])) <= 8 * R.U * 1.5 * float(dy[:, c].abs().sum())
