"""Layer calls on explicit streams without buffers of the caller's: the memory
of each call's workspace stays its own until its kernels are done, whatever
the current stream allocates meanwhile.  Results are bit-equal to those of the
same call alone."""
import numpy as np
import pytest
import torch

import synth
from fp8_block_scaled_pow2_b200.layer import MoeLayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call,shared", [("forward_few", "mxfp4"), ("forward", "mxfp4"), ("forward", "fp8")])
def test_calls_without_buffers_on_other_streams(lib, call, shared):
    H, I, E, k, T = 512, 256, 16, 4, 5
    G = E + 1
    w13, s13 = synth.quantize_mxfp4(synth.normal(31, 1, G * 2 * I * H).reshape(G * 2 * I, H) * 0.02)
    w2, s2 = synth.quantize_mxfp4(synth.normal(31, 2, G * H * I).reshape(G * H, I) * 0.02)
    layer = MoeLayer(w13.reshape(G, 2 * I, H // 2), s13.reshape(G, 2 * I, H // 32), w2.reshape(G, H, I // 2),
                     s2.reshape(G, H, I // 32), k, shared=shared)
    run = getattr(layer, call)
    ins = []
    for i in range(4):
        x = synth.to_bf16_bits(synth.normal(70 + i, 5, T * H).reshape(T, H)).view(np.int16)
        z = synth.normal(70 + i, 6, T * E).reshape(T, E).astype(np.float32)
        ins.append((torch.from_numpy(x).cuda(), torch.from_numpy(z).cuda()))
    ref = [run(x, z).clone() for x, z in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sizes = [lib.moe_layer_few_workspace_size(T, H, I, E, k), T * k * 4, T * H * 2]
    ys, junk = [], []
    for n in range(40):
        stream = streams[n % 2]
        ys.append(run(*ins[n % 4], stream=stream.cuda_stream if shared == "mxfp4" and n % 8 > 5 else stream))
        # memory of the current stream of the sizes that the call dropped, overwritten at once
        junk = [torch.full((b,), 0xFF, dtype=torch.uint8, device="cuda") for b in sizes]
    torch.cuda.synchronize()
    for n, y in enumerate(ys):
        assert torch.equal(y, ref[n % 4]), n
    # a result read on the current stream and dropped before it is read: its memory is not given to the next call
    torch.cuda.synchronize()
    got = []
    for n in range(40):
        y = run(*ins[n % 4], stream=streams[0])
        torch.cuda.current_stream().wait_stream(streams[0])
        got.append(y.float())
        del y
    torch.cuda.synchronize()
    for n, y in enumerate(got):
        assert torch.equal(y, ref[n % 4].float()), n
    assert lib.moe_get_device_error() == 0 and len(junk) == 3


@pytest.mark.parametrize("call", ["forward", "forward_few"])
def test_default_stream_handle_empty_batch_and_capture(lib, call):
    """The null handle names the default stream; no tokens; a captured call on
    a stream of its own, without buffers."""
    H, I, E, k, T = 256, 128, 8, 2, 3
    wl = synth.tiny_layer(2)
    layer = MoeLayer(wl.w13, wl.w13_e8m0, wl.w2, wl.w2_e8m0, k)
    run = getattr(layer, call)
    x = torch.from_numpy(wl.x_bf16[:T].view(np.int16)).cuda()
    z = torch.from_numpy(wl.logits[:T]).cuda()
    ref = run(x, z).clone()
    assert torch.equal(run(x, z, stream=0), ref)
    assert torch.equal(run(x, z, stream=torch.cuda.default_stream()), ref)
    side = torch.cuda.Stream()
    empty = torch.empty((0, H), dtype=torch.int16, device="cuda"), torch.empty((0, E), device="cuda")
    assert run(*empty, stream=side).shape == (0, H)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        y = run(x, z, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        out = y.clone()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert lib.moe_get_device_error() == 0
