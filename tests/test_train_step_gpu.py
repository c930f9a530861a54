"""The operators as a training step uses them: embedding, layer norm, an adapted
linear (the library's own forward and backward), layer norm's gradient, the
embedding's gradient, and the clipping of the factors' gradients. Against a
64-bit chain, eager and as a captured graph that is replayed on new inputs."""
import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from . import train_ops_reference as R
from .parity import dev, rel_fro

pytestmark = pytest.mark.gpu

T, V, N, D, RANK = 384, 500, 256, 320, 4


class Step:
    """One training step on fixed buffers; everything a call needs is kept."""

    def __init__(self, seed):
        g = torch.Generator(device=dev()).manual_seed(seed)
        r = lambda *s: torch.randn(*s, device=dev(), generator=g)
        e = lambda *s, dtype=torch.float32: torch.empty(*s, device=dev(), dtype=dtype)
        bf = torch.bfloat16
        self.table, self.ids = (0.02 * r(V, N)).to(bf), torch.randint(0, V, (T,), device=dev(), generator=g)
        self.weight, self.bias = 1 + 0.1 * r(N), 0.1 * r(N)
        self.W, self.A, self.Bm = (0.05 * r(D, N)).to(bf), (0.1 * r(D, RANK)).to(bf), (0.1 * r(RANK, N)).to(bf)
        self.dY = (1e-2 * r(T, D)).to(bf)
        self.h, self.x, self.Y = e(T, N), e(T, N, dtype=bf), e(T, D)
        self.mean, self.rstd = e(T), e(T)
        self.dx, self.dh = e(T, N), e(T, N)
        self.dA, self.dB = e(D, RANK), e(RANK, N)
        self.dweight, self.dbias, self.dtable, self.norm = e(N), e(N), e(V, N), e(1)
        self.emb = B.Descriptors([B.EmbeddingJob(self.table, self.ids, self.h, 16.0)])
        self.ln = B.Descriptors([B.LayerNormJob(self.h, self.weight, self.bias, self.x, self.mean, self.rstd)])
        self.lin = B.Descriptors([B.LinearJob(self.x, self.W, self.Y)])
        self.back = B.Descriptors([B.TrainBackwardJob(self.x, self.dY, self.W, self.A, self.Bm, self.dx, self.dA,
                                                      self.dB)])
        self.lnb = B.Descriptors([B.LayerNormBackwardJob(self.dx, self.h, self.weight, self.mean, self.rstd, self.dh,
                                                         self.dweight, self.dbias)])
        self.embb = B.Descriptors([B.EmbeddingBackwardJob(self.dh, self.ids, self.dtable, 16.0)])
        self.grads = B.Descriptors([B.GradJob(t) for t in (self.dA, self.dB, self.dweight, self.dbias, self.dtable)])
        size = lambda f, j: torch.empty(f(j), dtype=torch.uint8, device=dev())
        self.ws = [size(B.intlora_train_backward_workspace_size, self.back),
                   size(B.intlora_layer_norm_backward_workspace_size, self.lnb),
                   size(B.intlora_embedding_backward_workspace_size, self.embb),
                   size(B.intlora_grad_norm_workspace_size, self.grads)]

    def run(self):
        B.intlora_embedding_batched(self.emb)
        B.intlora_layer_norm_batched(self.ln)
        B.intlora_linear_bf16_batched(self.lin)
        B.intlora_train_backward_batched(self.back, self.ws[0])
        B.intlora_layer_norm_backward_batched(self.lnb, self.ws[1])
        B.intlora_embedding_backward_batched(self.embb, self.ws[2])
        B.intlora_clip_grad_norm_batched(self.grads, 0.5, self.norm, self.ws[3])

    def outputs(self):
        return dict(Y=self.Y, dA=self.dA, dB=self.dB, dweight=self.dweight, dbias=self.dbias, dtable=self.dtable,
                    norm=self.norm)

    def reference(self):
        """The same step in 64 bits, without the roundings between the calls."""
        h = R.embedding(self.table, self.ids, 16.0)
        x, mean, rstd = R.layer_norm(h, self.weight, self.bias, 1e-5)
        W, dY = self.W.double(), self.dY.double()
        G = dY.t() @ x
        dx = dY @ W
        dh, dweight, dbias = R.layer_norm_backward(dx, h, self.weight, mean, rstd)
        dtable, _, _ = R.embedding_backward(dh, self.ids, V, 16.0)
        out = dict(dA=G @ self.Bm.double().t(), dB=self.A.double().t() @ G, dweight=dweight, dbias=dbias, dtable=dtable)
        norm = R.grad_norm(list(out.values()))
        factor = min(1.0, 0.5 / (norm + 1e-6))
        assert factor < 0.9                        # the step does clip
        out = {k: v * factor for k, v in out.items()}
        return dict(out, Y=x @ W.t(), norm=torch.tensor([norm], dtype=torch.float64))


# x is rounded to bf16 once (half a step, 2^-8) on the way to Y, dA and dB; what
# else there is, is fp32 (the factors' gradients come from two exact bf16 halves,
# 2^-17). The clipped gradients also carry the norm's error, at most as large.
STEP_RTOL = 2 * 2.0 ** -8


def _check(step):
    ref = step.reference()
    for k, v in step.outputs().items():
        assert rel_fro(v.double().cpu().numpy(), ref[k].cpu().numpy()) < STEP_RTOL, k


def test_step_against_the_64_bit_chain():
    step = Step(1)
    step.run()
    _check(step)


def test_captured_step_replays_on_new_inputs():
    """Two steps captured into graphs of their own, each with its workspaces,
    replayed in turn, and one of them again on other inputs in its buffers."""
    steps = [Step(2), Step(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for s in steps:
            s.run()                                # first use outside the capture
        side.synchronize()
        for s in steps:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                s.run()
            graphs.append(g)
    for s in steps:
        for v in s.outputs().values():
            v.fill_(float("nan"))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for s in steps:
        _check(s)
    fresh = Step(4)
    for k in ("table", "ids", "weight", "bias", "W", "A", "Bm", "dY"):
        getattr(steps[0], k).copy_(getattr(fresh, k))
    graphs[0].replay()
    fresh.run()
    torch.cuda.synchronize()
    _check(steps[0])
    # the linear's backward adds split sums with atomics, so only what comes
    # before it, and through dX alone, has the same bits
    for a, b in ((steps[0].Y, fresh.Y), (steps[0].x, fresh.x), (steps[0].dh, fresh.dh)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two steps at once on two streams, each with its own workspaces."""
    steps = [Step(5), Step(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s in steps:
        _check(s)
