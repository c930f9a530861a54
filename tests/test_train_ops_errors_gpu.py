"""An error of one call does not show up in the next."""
import ctypes

import pytest
import torch

from quantized_lora_merge_b200 import binding as B

from .parity import dev

pytestmark = pytest.mark.gpu


def _refused_launch(call):
    """Runs `call` on a stream whose capture has been invalidated on the host (a
    capturing stream may not be synchronized): the launch is refused with an
    error code, and nothing reaches the GPU."""
    cuda = ctypes.CDLL("libcuda.so.1")
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(handle, 1) == 0
    try:
        assert cuda.cuStreamSynchronize(handle) != 0
        with pytest.raises(RuntimeError, match="launch"):
            call(side)
    finally:
        assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0


def _calls():
    g = torch.ones(1000, device=dev())
    norm = torch.ones(1, device=dev())
    x = torch.randn(4, 64, device=dev())
    y = torch.empty_like(x)
    ids = torch.zeros(4, dtype=torch.int64, device=dev())
    table = torch.zeros(9, 64, device=dev())
    mean, rstd = torch.zeros(4, device=dev()), torch.ones(4, device=dev())
    ln = B.LayerNormBackwardJob(x, x, None, mean, rstd, y)
    emb = B.EmbeddingBackwardJob(x, ids, table)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    return {
        "grad_norm of nothing": lambda s: B.intlora_grad_norm_batched([], norm, stream=s),
        "grad_norm": lambda s: B.intlora_grad_norm_batched([B.GradJob(g)], norm, ws, stream=s),
        "grad_clip": lambda s: B.intlora_grad_clip_batched([B.GradJob(g)], 1.0, norm, stream=s),
        "layer_norm": lambda s: B.intlora_layer_norm_batched([B.LayerNormJob(x, None, None, y)], stream=s),
        "layer_norm_backward": lambda s: B.intlora_layer_norm_backward_batched([ln], ws, stream=s),
        "embedding": lambda s: B.intlora_embedding_batched([B.EmbeddingJob(table, ids, y)], stream=s),
        "embedding_backward": lambda s: B.intlora_embedding_backward_batched([emb], ws, stream=s),
    }


@pytest.mark.parametrize("name", ["grad_norm of nothing", "grad_norm", "grad_clip", "layer_norm", "layer_norm_backward",
                                  "embedding", "embedding_backward"])
def test_a_refused_launch_leaves_no_error_behind(name):
    calls = _calls()
    torch.cuda.synchronize()
    _refused_launch(calls[name])
    for call in calls.values():                  # every first kernel is launched on a sound stream
        call(None)
    torch.cuda.synchronize()
