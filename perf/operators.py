"""Operators around the adapted linears of a training step, as they are measured.

Five operators stand beside the training forward and backward of the merged
linears (intlora_linear_bf16_batched, intlora_train_backward_batched):

  ln_fwd    layer norm over rows, the input of the linears
  ln_bwd    its gradients: dx, and dweight and dbias summed over all rows
  emb_fwd   embedding lookup with scaling, where the tokens enter
  emb_bwd   its gradient by sorted tokens: overwritten whole, or added to
  clip      global norm over the factors' gradients, and clipping in place

Where `own` is false, run() computes them in plain torch operations in 32 bits;
where it is true, it makes the library's calls. exact() has the same from the
definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
# widths of the SD-UNet-shaped transformer blocks, eight linears a block
UNET_WIDTHS = [320] * 2 + [640] * 2 + [1280] * 6 + [640] * 3 + [320] * 3
# the seven linears of a Llama-3-8B decoder layer, (d, n)
LLAMA_LINEARS = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096),
                 (14336, 4096), (14336, 4096), (4096, 14336)]


def listed():
    return [
        # one token through a norm at Llama-3-8B's width: latency alone counts
        dict(name="ln_fwd one token", op="ln_fwd", tokens=1, n=4096, x="bf16", p="bf16", y="bf16"),
        # four 64 x 64 latents in the widest-resolution UNet block, half precision
        dict(name="ln_fwd unet 320", op="ln_fwd", tokens=16384, n=320, x="f16", p="f32", y="f16"),
        # a ragged batch at an odd width, fp32 activations into the bf16 linears
        dict(name="ln_fwd odd rows", op="ln_fwd", tokens=1031, n=5003, x="f32", p="f32", y="bf16"),
        # 8192 tokens at Llama-3-8B's width: dy is the fp32 dX of the linears' backward
        dict(name="ln_bwd 8192x4096", op="ln_bwd", tokens=8192, n=4096, x="bf16", p="bf16", dy="f32", dx="f32"),
        # 16 x 16 latents of a batch in the deepest UNet blocks, all bf16
        dict(name="ln_bwd unet 1280", op="ln_bwd", tokens=4096, n=1280, x="bf16", p="f32", dy="bf16", dx="bf16"),
        # a small odd batch in fp32
        dict(name="ln_bwd odd rows", op="ln_bwd", tokens=333, n=1001, x="f32", p="f32", dy="f32", dx="f32"),
        # a decoding step of eight sequences
        dict(name="emb_fwd 8 tokens", op="emb_fwd", tokens=8, n=4096, vocab=32000, table="bf16", y="bf16",
             scale=1.0, zipf=1.0),
        # the tokens of a training step, scaled by the root of the width
        dict(name="emb_fwd 32768 tokens", op="emb_fwd", tokens=32768, n=4096, vocab=32000, table="bf16", y="bf16",
             scale=64.0, zipf=1.0),
        # a training step's gradient of the whole table, tokens by Zipf's law
        dict(name="emb_bwd whole table", op="emb_bwd", tokens=16384, n=4096, vocab=32000, dy="bf16", dtable="f32",
             scale=64.0, zipf=1.0, padding=False, accumulate=False),
        # four prompts of 77 tokens, padded, added to the gradient of a text encoder's table
        dict(name="emb_bwd prompts", op="emb_bwd", tokens=308, n=768, vocab=49408, dy="f32", dtable="f32",
             scale=1.0, zipf=1.0, padding=True, accumulate=True),
        # the 256 factor gradients of the UNet's 128 linears at rank 4
        dict(name="clip unet rank 4", op="clip", layers="unet", rank=4, blocks=16, g="f32", clip=0.5),
        # the 448 factor gradients of Llama-3-8B's 224 linears at rank 16
        dict(name="clip llama rank 16", op="clip", layers="llama", rank=16, blocks=32, g="f32", clip=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.35 else max(8, n // 8 * 8)     # odd widths among them


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "emb_fwd", "emb_bwd", "clip"])
    kind = lambda: rng.choice(["f32", "bf16", "f16"])
    if op in ("ln_fwd", "ln_bwd"):
        n = _width(rng, 64, 16384)
        tokens = _log_int(rng, 1, min(65536, 24_000_000 // n))
        if op == "ln_fwd":
            return dict(op=op, tokens=tokens, n=n, x=kind(), p=kind(), y=kind())
        return dict(op=op, tokens=tokens, n=n, x=kind(), p=kind(), dy=kind(), dx=kind())
    if op == "emb_fwd":
        n = _width(rng, 64, 8192)
        vocab = _log_int(rng, 100, min(131072, 130_000_000 // n))
        tokens = _log_int(rng, 1, min(65536, 60_000_000 // n))
        return dict(op=op, tokens=tokens, n=n, vocab=vocab, table=kind(), y=kind(),
                    scale=rng.choice([1.0, 0.5, math.sqrt(n)]), zipf=rng.choice([0.0, 1.0, 1.2]))
    if op == "emb_bwd":
        n = _width(rng, 64, 8192)
        vocab = _log_int(rng, 100, min(131072, 120_000_000 // n))
        tokens = _log_int(rng, 1, min(65536, 60_000_000 // n))
        return dict(op=op, tokens=tokens, n=n, vocab=vocab, dy=kind(), dtable="f32",
                    scale=rng.choice([1.0, 0.5, math.sqrt(n)]), zipf=rng.choice([0.0, 1.0, 1.2]),
                    padding=rng.random() < 0.5, accumulate=rng.random() < 0.5)
    layers = rng.choice(["unet", "llama"])
    return dict(op=op, layers=layers, rank=_log_int(rng, 1, 16), blocks=rng.randint(1, 16 if layers == "unet" else 32),
                g=kind(), clip=rng.choice([0.5, 0.1, 2.0]))


def _factor_shapes(case):
    """(rows, columns) of dA and dB of every adapted linear."""
    r = case["rank"]
    if case["layers"] == "llama":
        linears = LLAMA_LINEARS * case["blocks"]
    else:
        linears = [(d, n) for w in UNET_WIDTHS[:case["blocks"]]
                   for d, n in ((w, w), (w, w), (w, w), (w, w), (w, 768), (w, 768), (8 * w, w), (w, 4 * w))]
    return [shape for d, n in linears for shape in ((d, r), (r, n))]


def _randn(gen, *shape):
    return torch.randn(*shape, device=DEVICE, generator=gen)


def _ids(case, gen):
    """Token ids: Zipf's law over the vocabulary (exponent 0: uniform) in a
    shuffled order of words; the last tenth is the padding id where there is one."""
    V, T = case["vocab"], case["tokens"]
    weight = torch.arange(1, V + 1, device=DEVICE, dtype=torch.float64) ** -case["zipf"]
    cdf = torch.cumsum(weight, 0)
    u = torch.rand(T, device=DEVICE, generator=gen, dtype=torch.float64) * cdf[-1]
    rank = torch.searchsorted(cdf, u).clamp_(max=V - 1)
    ids = torch.randperm(V, device=DEVICE, generator=gen)[rank]
    if case.get("padding"):
        ids[T - T // 10:] = 0
    return ids


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op in ("ln_fwd", "ln_bwd"):
        T, n = case["tokens"], case["n"]
        # residual-stream activations: a spread of row scales and means, a few heavy channels
        x = _randn(gen, T, n) * torch.exp(0.5 * _randn(gen, T, 1)) + 0.3 * _randn(gen, T, 1)
        x[:, : max(1, n // 256)] *= 8
        s["x"] = x.to(TYPES[case["x"]])
        s["weight"] = (1 + 0.1 * _randn(gen, n)).to(TYPES[case["p"]])
        if op == "ln_fwd":
            s["bias"] = (0.1 * _randn(gen, n)).to(TYPES[case["p"]])
            s["y"] = torch.empty(T, n, device=DEVICE, dtype=TYPES[case["y"]])
            s["mean"] = torch.empty(T, device=DEVICE)
            s["rstd"] = torch.empty(T, device=DEVICE)
        else:
            # the statistics that the forward pass has left
            xd = s["x"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (xd.var(1, correction=0) + EPS).rsqrt().float()
            del xd
            s["dy"] = (0.02 * _randn(gen, T, n)).to(TYPES[case["dy"]])
            s["dx"] = torch.empty(T, n, device=DEVICE, dtype=TYPES[case["dx"]])
            s["dweight"] = torch.empty(n, device=DEVICE)
            s["dbias"] = torch.empty(n, device=DEVICE)
    elif op == "emb_fwd":
        s["table"] = (0.02 * _randn(gen, case["vocab"], case["n"])).to(TYPES[case["table"]])
        s["ids"] = _ids(case, gen)
        s["y"] = torch.empty(case["tokens"], case["n"], device=DEVICE, dtype=TYPES[case["y"]])
    elif op == "emb_bwd":
        s["dy"] = (0.02 * _randn(gen, case["tokens"], case["n"])).to(TYPES[case["dy"]])
        s["ids"] = _ids(case, gen)
        s["dtable"] = torch.empty(case["vocab"], case["n"], device=DEVICE, dtype=TYPES[case["dtable"]])
        if case["accumulate"]:
            s["dtable"].copy_(1e-3 * _randn(gen, case["vocab"], case["n"]))
    else:
        # one buffer for all gradients, each tensor at a 256-byte boundary
        kind = TYPES[case["g"]]
        item = 256 // torch.empty(0, dtype=kind).element_size()
        shapes = _factor_shapes(case)
        starts, total = [], 0
        for rows, cols in shapes:
            starts.append(total)
            total += (rows * cols + item - 1) // item * item
        flat = 0.01 * _randn(gen, total)
        used = torch.zeros(total, device=DEVICE)
        for at, (rows, cols) in zip(starts, shapes):
            used[at:at + rows * cols] = 1
        s["grads"] = (flat * used).to(kind)
        s["max_norm"] = float(case["clip"] * 0.01 * math.sqrt(sum(r * c for r, c in shapes)))
        s["norm"] = torch.empty(1, device=DEVICE)
        s["views"] = [s["grads"][at:at + rows * cols].view(rows, cols) for at, (rows, cols) in zip(starts, shapes)]
    if own:
        s.update(_plan(s))
    return s


def _plan(s):
    """What a program that repeats a step on the same buffers keeps: the
    descriptors and the workspace."""
    from quantized_lora_merge_b200 import binding as B
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        jobs = [B.LayerNormJob(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], EPS)]
        size = 0
    elif op == "ln_bwd":
        jobs = [B.LayerNormBackwardJob(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                       s["dbias"])]
        size = B.intlora_layer_norm_backward_workspace_size(jobs)
    elif op == "emb_fwd":
        jobs = [B.EmbeddingJob(s["table"], s["ids"], s["y"], case["scale"])]
        size = 0
    elif op == "emb_bwd":
        jobs = [B.EmbeddingBackwardJob(s["dy"], s["ids"], s["dtable"], case["scale"],
                                       padding_id=0 if case["padding"] else -1, accumulate=case["accumulate"])]
        size = B.intlora_embedding_backward_workspace_size(jobs)
    else:
        jobs = [B.GradJob(g) for g in s["views"]]
        size = B.intlora_grad_norm_workspace_size(jobs)
    return dict(B=B, jobs=B.Descriptors(jobs), ws=torch.empty(max(size, 256), device=DEVICE, dtype=torch.uint8))


def run(s):
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        if own:
            s["B"].intlora_layer_norm_batched(s["jobs"])
            return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
        y = xc * rstd * s["weight"].float() + s["bias"].float()
        return dict(y=y.to(s["y"].dtype), mean=mean[:, 0], rstd=rstd[:, 0])
    if op == "ln_bwd":
        if own:
            s["B"].intlora_layer_norm_backward_batched(s["jobs"], s["ws"])
            return dict(dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])
        dy = s["dy"].float()
        rstd = s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        return dict(dx=dx.to(s["dx"].dtype), dweight=(dy * xhat).sum(0), dbias=dy.sum(0))
    if op == "emb_fwd":
        if own:
            s["B"].intlora_embedding_batched(s["jobs"])
            return dict(y=s["y"])
        return dict(y=(s["table"][s["ids"]].float() * case["scale"]).to(s["y"].dtype))
    if op == "emb_bwd":
        if own:
            s["B"].intlora_embedding_backward_batched(s["jobs"], s["ws"])
            return dict(dtable=s["dtable"])
        dy = s["dy"].float() * case["scale"]
        if case["padding"]:
            dy = dy * (s["ids"] != 0)[:, None]
        if not case["accumulate"]:
            s["dtable"].zero_()
        return dict(dtable=s["dtable"].index_add_(0, s["ids"], dy))
    if own:
        s["B"].intlora_clip_grad_norm_batched(s["jobs"], s["max_norm"], s["norm"], s["ws"])
        return dict(grads=s["grads"], norm=s["norm"])
    g = s["grads"].float()
    norm = (g * g).sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    s["grads"].copy_(g * scale)
    return dict(grads=s["grads"], norm=norm[None])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = 1.0 / torch.sqrt(var + EPS)
        return dict(y=torch.addcmul(s["bias"].double(), (x - mean) * rstd, s["weight"].double()),
                    mean=mean.squeeze(1), rstd=rstd.squeeze(1))
    if op == "ln_bwd":
        n = case["n"]
        mean, rstd = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1)
        dy, xhat = s["dy"].double(), (s["x"].double() - mean).mul_(rstd)
        w = s["weight"].double()
        c1 = dy @ w / n                                     # row means of dy w and of dy w xhat
        c2 = torch.einsum("tn,tn,n->t", dy, xhat, w) / n
        dweight, dbias = torch.einsum("tn,tn->n", dy, xhat), torch.einsum("tn->n", dy)
        dx = rstd * (dy * w - c1.unsqueeze(1) - c2.unsqueeze(1) * xhat)
        return dict(dx=dx, dweight=dweight, dbias=dbias)
    if op == "emb_fwd":
        return dict(y=s["table"].double().index_select(0, s["ids"]).mul_(case["scale"]))
    if op == "emb_bwd":
        # sums of runs of equal tokens, by differences of the running sum over the sorted tokens
        ids, order = torch.sort(s["ids"], stable=True)
        run = torch.cumsum(s["dy"].double().index_select(0, order), 0)
        last = torch.ones_like(ids, dtype=torch.bool)
        last[:-1] = ids[1:] != ids[:-1]
        ends = run[last]
        sums = ends.clone()
        sums[1:] -= ends[:-1]
        words = ids[last]
        if case["padding"]:
            sums[words == 0] = 0
        out = s["dtable"].double() if case["accumulate"] else torch.zeros(s["dtable"].shape, device=DEVICE,
                                                                          dtype=torch.float64)
        out[words] += case["scale"] * sums
        return dict(dtable=out)
    g = s["grads"].double()
    norm = torch.sqrt(torch.dot(g, g))
    return dict(grads=g * min(1.0, s["max_norm"] / (float(norm) + 1e-6)), norm=norm.reshape(1))


def work(case):
    """Bytes: every input read once and every output written once."""
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op in ("ln_fwd", "ln_bwd"):
        T, n = case["tokens"], case["n"]
        if op == "ln_fwd":
            return dict(bytes=T * n * (size[case["x"]] + size[case["y"]]) + 2 * n * size[case["p"]] + 8 * T,
                        flops=8 * T * n)
        return dict(bytes=T * n * (size[case["x"]] + size[case["dy"]] + size[case["dx"]]) + n * size[case["p"]] + 8 * T
                    + 8 * n, flops=14 * T * n)
    if op == "emb_fwd":
        T, n = case["tokens"], case["n"]
        rows = _expected_words(case)        # a row that several tokens read comes from memory once
        return dict(bytes=rows * n * size[case["table"]] + T * n * size[case["y"]] + 8 * T, flops=T * n)
    if op == "emb_bwd":
        T, n = case["tokens"], case["n"]
        rows = _expected_words(case)
        moved = 2 * rows if case["accumulate"] else case["vocab"]
        return dict(bytes=T * n * size[case["dy"]] + moved * n * size[case["dtable"]] + 8 * T, flops=T * n)
    count = sum(r * c for r, c in _factor_shapes(case))
    return dict(bytes=count * size[case["g"]] * (2 if case["clip"] < 1 else 1), flops=3 * count)


def _expected_words(case):
    """Distinct words among the tokens, expected under the law they are drawn from."""
    V, T, a = case["vocab"], case["tokens"], case["zipf"]
    weight = torch.arange(1, V + 1, dtype=torch.float64) ** -a
    return float((1 - (1 - weight / weight.sum()) ** T).sum())
