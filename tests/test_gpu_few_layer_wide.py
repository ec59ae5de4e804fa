"""The few-token layer at the ends of its range: every width of the routing
(256, 512 and 1024 experts), the longest list of chosen experts, the widest
rows with a few ring slots, and the decode size with a full batch.

Tolerances of y: those of the layer's other paths (see test_gpu_few_layer)."""
import numpy as np
import pytest
import torch

import synth
from fp8_block_scaled_pow2_b200.layer import MoeLayer
from oracle import ffn
from tests.test_gpu_few_layer import check_y, dev, inputs

pytestmark = pytest.mark.gpu


class Few:
    """A layer whose experts share a few prototypes (every expert has its own memory on the device)."""

    def __init__(self, seed, H, I, E, n_proto, k, shared=1, tid2eid=None):
        self.E, self.k, self.shared, self.tid2eid = E, k, shared, tid2eid
        self.w = synth.expert_views(seed, E + shared, H, I, n_proto)
        w13, s13, w2, s2 = self.w
        self.layer = MoeLayer(w13[:], s13[:], w2[:], s2[:], k, has_shared=shared, tid2eid=tid2eid)

    def ref(self, xb, z, tok=None):
        w13, s13, w2, s2 = self.w
        return ffn.moe_layer(xb, z, w13, s13, w2, s2, self.k, has_shared=self.shared, cache={}, token_ids=tok,
                             tid2eid=self.tid2eid)

    def run(self, xb, z, tok=None):
        T = xb.shape[0]
        buf = self.layer.alloc_few(T)
        for t in (buf.idx, buf.w, buf.y):
            t.fill_(-7)
        buf.workspace.fill_(0xFF)
        self.layer.forward_few(dev(xb.view(np.int16)), dev(z), buf, token_ids=None if tok is None else dev(tok))
        return buf


@pytest.mark.parametrize("E", [255, 256, 257, 384, 511, 512, 513, 1024])
@pytest.mark.parametrize("T,k", [(1, 6), (16, 6), (16, 16)])
def test_routing_widths(lib, E, T, k):
    """Winners among the last experts, and ties across the borders of the
    routing's register blocks."""
    c = Few(E, 256, 128, E, 5, k)
    xb, z = inputs(E + T, T, 256, E)
    z[0, -1] = 9                                             # the last expert wins
    if T > 1:
        z[1, -k:] = 5 + np.arange(k)                         # all winners at the end
        z[2] = 0.5                                           # one tie over all experts
        z[3, :] = np.minimum(z[3], 3)
        z[3, [i for i in (31, 32, 255, 256, 511, 512, E - 1) if i < E]] = 4      # ties across the borders
        z[4, E // 2:] = -np.inf
        z[5, 1::2] = np.finfo(np.float32).min
    buf = c.run(xb, z)
    ref = c.ref(xb, np.maximum(z, -1e30))
    np.testing.assert_array_equal(buf.idx.cpu().numpy(), ref["idx"])
    i2, w2 = torch.empty_like(buf.idx), torch.empty_like(buf.w)
    lib.moe_route_topk(dev(z), k, i2, w2)
    assert torch.equal(buf.idx, i2) and torch.equal(buf.w, w2)
    check_y(buf.y, ref["y"])
    assert lib.moe_get_device_error() == 0


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("hashed", [False, True])
@pytest.mark.parametrize("E", [256, 1024])
def test_longest_list(lib, shared, hashed, E):
    """16 tokens with 16 experts each, all different: 256 entries, and the
    shared expert."""
    T, k = 16, 16
    order = np.argsort(synth.uniform(E, 9, E), kind="stable")
    picks = order[:T * k].reshape(T, k).astype(np.int32)
    table = tok = None
    xb, z = inputs(E + shared, T, 256, E)
    if hashed:
        table = np.concatenate([picks[::-1], picks[:3]])     # token t has row 15 - t
        tok = (15 - np.arange(T)).astype(np.int32)
    else:
        np.put_along_axis(z, picks, np.abs(np.take_along_axis(z, picks, 1)) + 8, axis=1)
    c = Few(E + 1, 256, 128, E, 7, k, shared, table)
    buf = c.run(xb, z, tok)
    ref = c.ref(xb, z, tok)
    np.testing.assert_array_equal(buf.idx.cpu().numpy(), ref["idx"])
    assert len(np.unique(ref["idx"])) == T * k
    check_y(buf.y, ref["y"])
    assert lib.moe_get_device_error() == 0


@pytest.mark.parametrize("T,H,I", [(9, 7168, 2048), (16, 7168, 1024), (16, 8192, 2048), (12, 8064, 896), (8, 8192, 1024)])
def test_wide_rows_with_few_ring_slots(lib, T, H, I):
    c = Few(H + T, H, I, 6, 2, 3)
    xb, z = inputs(H + T, T, H, 6)
    buf = c.run(xb, z)
    ref = c.ref(xb, z)
    np.testing.assert_array_equal(buf.idx.cpu().numpy(), ref["idx"])
    check_y(buf.y, ref["y"])
    again = c.run(xb, z)
    assert torch.equal(buf.y, again.y) and lib.moe_get_device_error() == 0


@pytest.mark.parametrize("T", [11, 16])
def test_decode_size_full_batch(lib, T):
    """Hidden 4096, intermediate 2048, 384 + 1 experts, top-6."""
    c = Few(41, 4096, 2048, 384, 3, 6)
    xb, z = inputs(42 + T, T, 4096, 384)
    buf = c.run(xb, z)
    ref = c.ref(xb, z)
    np.testing.assert_array_equal(buf.idx.cpu().numpy(), ref["idx"])
    check_y(buf.y, ref["y"])
    assert lib.moe_get_device_error() == 0
