"""Refusals and sizes of the few-token layer and the 4-bit matrix-vector
products, without a GPU: every check below returns before any CUDA call."""
import ctypes

import pytest
import torch

from fp8_block_scaled_pow2_b200 import _lib, moe

OK, INVALID, UNSUPPORTED = 0, -1, -2
A = 1 << 20          # a well aligned address that a refused call never touches


def few(T=1, H=256, I=128, E=8, topk=2, x=A, logits=A, token_ids=None, tid2eid=None, vocab=0, w13=A, w2=A, idx=A, w=A,
        y=A, ws=A, ws_bytes=1 << 20, cfg=True):
    c = _lib.MoeConfig(T, H, I, E, topk, 1.5, 10.0, 1, 1)
    return _lib.load().moe_layer_few_mxfp4(ctypes.byref(c) if cfg else None, x, logits, token_ids, tid2eid, vocab, w13,
                                           w2, idx, w, y, ws, ws_bytes, None)


def test_few_workspace_size():
    size = moe.moe_layer_few_workspace_size
    assert size(1, 4096, 2048, 256, 6) >= 7 * 2048 and size(1, 4096, 2048, 256, 6) % 256 == 0
    assert size(16, 4096, 2048, 256, 6, 0) >= 96 * 2048
    assert size(0, 256, 128, 8, 2) > 0                     # an empty batch is valid
    for bad in ((17, 256, 128, 8, 2), (-1, 256, 128, 8, 2), (1, 200, 128, 8, 2), (1, 256, 100, 8, 2),
                (1, 256, 128, 0, 2), (1, 256, 128, 1025, 2), (1, 256, 128, 8, 0), (1, 256, 128, 32, 17),
                (1, 8320, 128, 8, 2), (1, 256, 8320, 8, 2)):
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("kw,status", [
    (dict(cfg=False), INVALID), (dict(T=0), OK), (dict(T=-1), INVALID), (dict(T=17), UNSUPPORTED),
    (dict(H=8320), UNSUPPORTED), (dict(I=8320), UNSUPPORTED), (dict(H=192), INVALID), (dict(I=0), INVALID),
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(topk=0), INVALID), (dict(topk=9), INVALID),
    (dict(topk=17, E=64), INVALID), (dict(x=None), INVALID), (dict(logits=None), INVALID), (dict(w13=None), INVALID),
    (dict(w2=None), INVALID), (dict(idx=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(x=A + 8), INVALID), (dict(w13=A + 16), INVALID),
    (dict(w2=A + 16), INVALID), (dict(ws=A + 16), INVALID), (dict(y=A + 2), INVALID), (dict(logits=A + 2), INVALID),
    (dict(token_ids=A, vocab=5), INVALID), (dict(tid2eid=A, vocab=5), INVALID),
    (dict(token_ids=A, tid2eid=A, vocab=0), INVALID), (dict(T=0, token_ids=A, tid2eid=A, vocab=5, topk=9), OK),
])
def test_few_refusals(kw, status):
    assert few(**kw) == status


def mv(fn, x=A, xt=1, ldx=128, M=1, w=A, s=A, g=A, N=8, K=128, out=A, ot=1, ldo=8):
    args = [x, xt, ldx, M, w, s] + ([g] if fn == "moe_matvec_nvfp4" else []) + [N, K, out, ot, ldo, None]
    return getattr(_lib.load(), fn)(*args)


@pytest.mark.parametrize("fn", ["moe_matvec_mxfp4", "moe_matvec_nvfp4", "moe_matvec_int4g128"])
@pytest.mark.parametrize("kw,status", [
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(M=17), UNSUPPORTED),
    (dict(K=32896, ldx=32896), UNSUPPORTED), (dict(K=0, ldx=8), INVALID), (dict(K=48), INVALID), (dict(xt=3), INVALID), (dict(ot=-1), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(s=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=127), INVALID), (dict(ldo=7), INVALID), (dict(w=A + 8), INVALID), (dict(x=A + 1), INVALID),
    (dict(out=A + 2, ot=0), INVALID), (dict(N=2 ** 31 - 1, ldo=2 ** 31 - 1), UNSUPPORTED),
])
def test_matvec_refusals(fn, kw, status):
    assert mv(fn, **kw) == status


def test_matvec_format_refusals():
    assert mv("moe_matvec_int4g128", K=96) == INVALID            # whole groups of 128
    assert mv("moe_matvec_int4g128", s=A + 2) == INVALID
    assert mv("moe_matvec_nvfp4", g=None) == INVALID
    assert mv("moe_matvec_nvfp4", g=A + 2) == INVALID


def test_binding_refuses_another_device():
    class On:
        def __init__(self, dev):
            self.dev = dev

        def get_device(self):
            return self.dev

    moe._one_device(1, On(1), None, On(1))
    with pytest.raises(ValueError):
        moe._one_device(1, On(1), On(0))


def test_binding_refuses_mismatched_tensors():
    """Shapes and types that do not belong together are refused before the call."""
    x, out = torch.zeros(2, 256), torch.zeros(2, 8)
    w, s = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(8, 8, dtype=torch.uint8)
    for bad in ((x[:, :128], w, s, out), (x, w, s[:, :7], out), (x, w, s, out[:, :7]), (x, w, s.float(), out),
                (x, w, s, out[:1])):
        with pytest.raises(ValueError):
            moe.moe_matvec_mxfp4(*bad)
    with pytest.raises(ValueError):
        moe.moe_matvec_mxfp4(x, w, s, out)                       # tensors that are not on a GPU
    with pytest.raises(ValueError):
        moe.moe_matvec_nvfp4(x, w, torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(2), out)
    with pytest.raises(ValueError):
        moe.moe_matvec_int4g128(x, w.view(torch.int8), torch.zeros(8, 2, dtype=torch.float64), out)
    T, H, I, E, k = 2, 256, 128, 8, 2
    p13 = torch.zeros(moe.moe_prepared_weights_size(E + 1, 2 * I, H), dtype=torch.uint8)
    p2 = torch.zeros(moe.moe_prepared_weights_size(E + 1, H, I), dtype=torch.uint8)
    good = dict(x=torch.zeros(T, H, dtype=torch.bfloat16), logits=torch.zeros(T, E), w13_prepared=p13, w2_prepared=p2,
                I=I, idx=torch.zeros(T, k, dtype=torch.int32), w=torch.zeros(T, k),
                y=torch.zeros(T, H, dtype=torch.bfloat16), workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    for bad in (dict(logits=torch.zeros(1, E)), dict(y=torch.zeros(T, H)), dict(idx=torch.zeros(T, k)),
                dict(w=torch.zeros(T, k + 1)), dict(has_shared=0), dict(I=256), dict(x=torch.zeros(T, H)),
                dict(token_ids=torch.zeros(T, dtype=torch.int32)), dict(tid2eid=torch.zeros(5, k, dtype=torch.int32)),
                dict(token_ids=torch.zeros(T, dtype=torch.int64), tid2eid=torch.zeros(5, k, dtype=torch.int32)), {}):
        with pytest.raises(ValueError):
            moe.moe_layer_few_mxfp4(**(good | bad))
