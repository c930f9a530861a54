"""Sums of the embedding and layer norm gradients that are exact in fp32: small
whole numbers and scales that are powers of two. Every order of addition gives
the same bits, so that a token or row that is lost or counted twice shows, of
however many; bounds that grow with the number of terms cannot show that."""
import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from .parity import dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _whole(gen, most, *shape):
    return torch.randint(-most, most + 1, shape, device=dev(), generator=gen)


def _embedding_gradient(dy, ids, vocab, scale, old, dtype=F32):
    dtable = torch.full((vocab, dy.shape[1]), 77.0, device=dev(), dtype=dtype) if old is None else old.to(dtype)
    jobs = [B.EmbeddingBackwardJob(dy, ids, dtable, scale, accumulate=old is not None)]
    ws = torch.empty(max(1, B.intlora_embedding_backward_workspace_size(jobs)), dtype=torch.uint8, device=dev())
    B.intlora_embedding_backward_batched(jobs, ws)
    return dtable


def _law(law, tokens, vocab, gen):
    if law == "one word":
        return torch.full((tokens,), vocab // 2, device=dev())
    if law == "half":                            # one word has every other token
        ids = torch.randint(0, vocab, (tokens,), device=dev(), generator=gen)
        ids[::2] = vocab - 1
        return ids
    return torch.randint(0, vocab, (tokens,), device=dev(), generator=gen)


# |sums| stay below 2^24: 3 x 2^21 tokens at most
@pytest.mark.parametrize("tokens", [48, 49, 511, 512, 513, 544, 4097, 16383, 16384, 16385, 40000])
@pytest.mark.parametrize("law,vocab", [("one word", 40), ("half", 300), ("uniform", 7), ("uniform", 30000)])
@pytest.mark.parametrize("n,dtype", [(8, F32), (24, BF16), (301, F16), (264, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_loses_no_token(tokens, law, vocab, n, dtype, accumulate):
    gen = torch.Generator(device=dev()).manual_seed(tokens + n)
    dy = _whole(gen, 3, tokens, n)
    ids = _law(law, tokens, vocab, gen)
    old = _whole(gen, 9, vocab, n) if accumulate else None
    want = torch.zeros(vocab, n, device=dev(), dtype=torch.int64).index_add_(0, ids, dy)
    got = _embedding_gradient(dy.to(dtype), ids, vocab, 0.5, None if old is None else old.float())
    assert torch.equal(got.double(), want * 0.5 + (0 if old is None else old))


@pytest.mark.parametrize("tokens", [2**20 - 1, 2**20, 2**20 + 1, 2**20 + 2**14 + 5])
@pytest.mark.parametrize("law,vocab", [("one word", 5000), ("half", 5000), ("uniform", 50), ("uniform", 2**21)])
@pytest.mark.parametrize("n", [1, 8])
def test_embedding_gradient_of_long_texts(tokens, law, vocab, n):
    """Around 2^20 tokens, where a third level of joins begins."""
    gen = torch.Generator(device=dev()).manual_seed(tokens + n)
    dy = _whole(gen, 3, tokens, n)
    ids = _law(law, tokens, vocab, gen)
    want = torch.zeros(vocab, n, device=dev(), dtype=torch.int64).index_add_(0, ids, dy)
    assert torch.equal(_embedding_gradient(dy.float(), ids, vocab, 2.0, None).double(), want * 2.0)


# ring places used again and again, rows shorter than an access, teams of every
# width, and rows too wide for registers
SHAPES = [(6000, n) for n in (1, 2, 3, 5, 7, 8, 12, 40)] + [
    (1300, 33), (700, 320), (4096, 1280), (333, 1001), (1300, 1001), (500, 4096), (300, 5003), (600, 9000), (151, 16384),
    (20, 40000), (300, 24576), (1, 64), (0, 64)]


@pytest.mark.parametrize("tokens,n", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift", [0, 1, 3, 6])
@pytest.mark.parametrize("accumulate", [False, True])
def test_layer_norm_gradient_loses_no_row(tokens, n, dtype, shift, accumulate):
    """With mean 0 and rstd 1, dweight is the sum of dy x and dbias that of dy."""
    gen = torch.Generator(device=dev()).manual_seed(tokens + n)
    x, dy = (torch.empty(tokens * n + shift, device=dev(), dtype=dtype)[shift:].view(tokens, n) for _ in range(2))
    xi, di = _whole(gen, 2, tokens, n), _whole(gen, 3, tokens, n)
    x.copy_(xi)
    dy.copy_(di)
    old = _whole(gen, 9, 2, n) if accumulate else torch.zeros(2, n, device=dev())
    dw, db = (old.float().clone() if accumulate else torch.full((2, n), 77.0, device=dev())).unbind(0)
    mean, rstd = torch.zeros(tokens, device=dev()), torch.ones(tokens, device=dev())
    for dx in (torch.empty(tokens, n, device=dev()), None):
        dw2, db2 = dw.clone(), db.clone()
        jobs = [B.LayerNormBackwardJob(dy, x, None, mean, rstd, dx, dw2, db2, accumulate)]
        ws = torch.empty(max(1, B.intlora_layer_norm_backward_workspace_size(jobs)), dtype=torch.uint8, device=dev())
        B.intlora_layer_norm_backward_batched(jobs, ws)
        assert torch.equal(dw2.double(), (di * xi).sum(0) + old[0].double())
        assert torch.equal(db2.double(), di.sum(0) + old[1].double())
