"""Timed cases of the operators for a handful of tokens.

Two operators, each in a plain form and as the library's call:

layer   one whole MoE layer step for T <= 16 tokens with MXFP4 experts
        (moe_layer_few_mxfp4): activation quantisation, routing, the gate / up
        products of the chosen experts, SwiGLU, requantisation, the down
        product and the weighted sum.
matvec  y[m, n] = sum_k x[m, k] * w[n, k] for M <= 16 rows and one 4-bit weight
        matrix with group scales: MXFP4 (moe_matvec_mxfp4), NVFP4
        (moe_matvec_nvfp4) or symmetric INT4 group-128 (moe_matvec_int4g128).

The plain forms compute in float32 with elementary tensor operations and
round once at the end (and where the layer itself quantises).
"""
import math

import torch

own = False

LIMIT = 10.0          # SwiGLU clamp
ROUTE_SCALE = 1.5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WEIGHT_SIGMA = 0.02


# --------------------------------- cases -----------------------------------
def _layer(name, T, H, I, E, topk, shared=True, hashed=False, norm=True):
    return {"name": name, "op": "layer", "T": T, "H": H, "I": I, "E": E, "topk": topk, "shared": shared,
            "hashed": hashed, "norm": norm}


def _matvec(name, fmt, M, N, K, x, out):
    return {"name": name, "op": "matvec", "fmt": fmt, "M": M, "N": N, "K": K, "x": x, "out": out}


def listed():
    return [
        # the smallest configuration: 16 tokens through 8 + 1 small experts, where only latency counts
        _layer("layer_tiny_t16", 16, 256, 128, 8, 2),
        # one decoded token of one sequence through the 256-expert layer
        _layer("layer_t1", 1, 4096, 2048, 256, 6),
        # a small batch (or a few drafted tokens) through the same layer
        _layer("layer_t4", 4, 4096, 2048, 256, 6),
        # the largest: 16 sequences decoding through the 384-expert variant
        _layer("layer_t16_e384", 16, 4096, 2048, 384, 6),
        # odd sizes, hash routing (the first layers), no shared expert, weights not normalised
        _layer("layer_hash_t3", 3, 1408, 640, 40, 3, shared=False, hashed=True, norm=False),
        # smallest matvec: a ragged head of a small model, float32 activations
        _matvec("mv_mxfp4_small_f32", "mxfp4", 2, 513, 160, "f32", "f32"),
        # one token times the w2 matrix of one expert, float32 result for a weighted sum
        _matvec("mv_mxfp4_t1", "mxfp4", 1, 4096, 2048, "bf16", "f32"),
        # one token times the stacked w1 | w3 matrix of one expert in INT4
        _matvec("mv_int4_t1", "int4", 1, 4096, 4096, "bf16", "bf16"),
        # a few tokens times an NVFP4 matrix in half precision
        _matvec("mv_nvfp4_t4_f16", "nvfp4", 4, 4096, 4096, "f16", "f16"),
        # odd row counts on both sides
        _matvec("mv_int4_ragged", "int4", 7, 5003, 1408, "f16", "f32"),
        # a large projection (16 stacked w1 | w3 matrices) for a batch of 8
        _matvec("mv_mxfp4_large_t8", "mxfp4", 8, 65536, 4096, "bf16", "bf16"),
        # the largest matrix, one token: a stream of weights and nothing else
        _matvec("mv_nvfp4_large_t1", "nvfp4", 1, 131072, 4096, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    if rng.random() < 0.5:
        E = rng.choice([8, 16, 40, 64, 128, 256, 384])
        return {k: v for k, v in _layer(
            "", _log(rng, 1, 16), 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 16), E, rng.randint(1, min(8, E)),
            shared=rng.random() < 0.7, hashed=rng.random() < 0.3, norm=rng.random() < 0.8).items() if k != "name"}
    fmt = rng.choice(["mxfp4", "nvfp4", "int4"])
    K = 128 * _log(rng, 1, 64) if fmt == "int4" or rng.random() < 0.5 else 32 * _log(rng, 1, 256)
    N = _log(rng, 1, min(131072, 400_000_000 // K))
    return {k: v for k, v in _matvec("", fmt, rng.randint(1, 16), N, K, rng.choice(["bf16", "bf16", "f16", "f32"]),
                                     rng.choice(["bf16", "f16", "f32"])).items() if k != "name"}


def _distinct(case):
    """Expected number of routed experts that T tokens with uniform routing reach."""
    return case["E"] * (1.0 - (1.0 - case["topk"] / case["E"]) ** case["T"])


def work(case):
    if case["op"] == "layer":
        T, H, I, k = case["T"], case["H"], case["I"], case["topk"]
        expert = 3 * H * I / 2 * 17 / 16                     # nibbles + one scale byte per 32
        n = _distinct(case) + (1 if case["shared"] else 0)
        io = T * H * 2 * 2 + T * (case["E"] * 4 if not case["hashed"] else k * 8) + T * k * 8
        return {"bytes": n * expert + io, "flops": 2.0 * 3 * H * I * T * (k + (1 if case["shared"] else 0))}
    M, N, K = case["M"], case["N"], case["K"]
    scale = {"mxfp4": 1 / 32, "nvfp4": 1 / 16, "int4": 4 / 128}[case["fmt"]]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    return {"bytes": N * K * (0.5 + scale) + M * K * size[case["x"]] + M * N * size[case["out"]],
            "flops": 2.0 * M * N * K}


# --------------------------------- inputs ----------------------------------
def _generator(case, seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1_000_003 + 17)


def _mxfp4(g, n, N, K):
    """Weights N(0, 0.02) as MXFP4: nibbles uint8 [n, N, K/2], E8M0 uint8 [n, N, K/32]."""
    nib = torch.empty((n, N, K // 2), dtype=torch.uint8, device="cuda")
    sc = torch.empty((n, N, K // 32), dtype=torch.uint8, device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, 33_554_432 // (N * K))
    rows = N if N * K <= 33_554_432 else max(1, 33_554_432 // K)
    for a in range(0, n, step):
        b = min(n, a + step)
        for r in range(0, N, rows):
            s = min(N, r + rows)
            w = torch.randn((b - a, s - r, K // 32, 32), device="cuda", generator=g) * WEIGHT_SIGMA
            e = torch.ceil(torch.log2(w.abs().amax(-1) / 6.0)).clamp_(-127, 127)
            v = w * torch.exp2(-e).unsqueeze(-1)
            code = torch.bucketize(v.abs(), mid, out_int32=True) + (v < 0) * 8
            code = code.to(torch.uint8).view(b - a, s - r, K // 2, 2)
            nib[a:b, r:s] = code[..., 0] | (code[..., 1] << 4)
            sc[a:b, r:s] = (e + 127).to(torch.uint8)
    return nib, sc


def prepare(case, seed):
    g = _generator(case, seed)
    if case["op"] == "layer":
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["topk"]
        G = E + (1 if case["shared"] else 0)
        x = torch.randn((T, H), device="cuda", generator=g)
        x = torch.where(torch.rand((T, H), device="cuda", generator=g) < 1e-3, x * 20, x)   # outlier channels
        st = {"case": case, "x": x.to(torch.bfloat16), "logits": torch.randn((T, E), device="cuda", generator=g)}
        if case["hashed"]:
            vocab = 1000
            st["tid2eid"] = torch.rand((vocab, E), device="cuda", generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
            st["token_ids"] = torch.randint(0, vocab, (T,), device="cuda", generator=g, dtype=torch.int32)
        st["w13"], st["w13_scale"] = _mxfp4(g, G, 2 * I, H)
        st["w2"], st["w2_scale"] = _mxfp4(g, G, H, I)
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        if own:
            # what a program keeps: the weights in the order the library's kernels stream, and scratch
            from fp8_block_scaled_pow2_b200 import moe
            for name, N, K, paired in (("w13", 2 * I, H, True), ("w2", H, I, False)):
                st[name + "_p"] = torch.empty(moe.moe_prepared_weights_size(G, N, K), dtype=torch.uint8, device="cuda")
                moe.moe_prepare_weights(st[name], st[name + "_scale"], st[name + "_p"], paired=paired)
            n = moe.moe_layer_few_workspace_size(T, H, I, E, k, int(case["shared"]))
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return st
    M, N, K, fmt = case["M"], case["N"], case["K"], case["fmt"]
    x = torch.randn((M, K), device="cuda", generator=g)
    x = torch.where(torch.rand((M, K), device="cuda", generator=g) < 1e-3, x * 20, x)
    st = {"case": case, "x": x.to(DTYPES[case["x"]]),
          "out": torch.empty((M, N), dtype=DTYPES[case["out"]], device="cuda")}
    if fmt == "int4":
        q = torch.empty((N, K // 2), dtype=torch.int8, device="cuda")
        sc = torch.empty((N, K // 128), dtype=torch.float32, device="cuda")
        rows = max(1, 33_554_432 // K)
        for r in range(0, N, rows):
            s = min(N, r + rows)
            w = torch.randn((s - r, K // 128, 128), device="cuda", generator=g) * WEIGHT_SIGMA
            sc[r:s] = w.abs().amax(-1) / 7.0
            c = torch.round(w / sc[r:s].unsqueeze(-1)).to(torch.int32).view(s - r, K // 2, 2) & 15
            q[r:s] = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8).view(torch.int8)
        st["w"], st["scale"] = q, sc
    else:
        nib, sc = _mxfp4(g, 1, N, K)
        st["w"], st["scale"] = nib[0], sc[0]
        if fmt == "nvfp4":
            # two E4M3 scales per 32 weights that differ, and one float32 factor for the matrix
            s = torch.rand((N, K // 16), device="cuda", generator=g) * 240 + 16
            st["scale"] = s.to(torch.float8_e4m3fn).view(torch.uint8)
            st["global"] = torch.rand(1, device="cuda", generator=g) * 1e-4 + 1e-5
    return st


# ------------------------------- plain forms --------------------------------
def _nibbles(packed):
    """uint8 [..., n] -> int32 codes [..., 2n], the low nibble first."""
    p = packed.to(torch.int32)
    return torch.stack((p & 15, (p >> 4) & 15), -1).flatten(-2)


def _fp4(packed):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=packed.device)
    return table[_nibbles(packed)]


def _mx_dequant(packed, e8m0):
    w = _fp4(packed)
    s = torch.ldexp(torch.ones((), device=w.device), e8m0.to(torch.int32) - 127)
    return (w.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _quantise(x):
    """Per 128 columns: E4M3 codes times their power-of-two scale, as float32."""
    g = x.unflatten(-1, (-1, 128))
    amax = g.abs().amax(-1)
    mant, ex = torch.frexp(amax / 448.0)
    k = torch.where(mant > 0.5, ex, ex - 1).clamp(-127, 127)
    k = torch.where(amax > 0, k, torch.zeros_like(k)).unsqueeze(-1)
    q = torch.ldexp(g, -k).clamp(-448, 448).to(torch.float8_e4m3fn).to(torch.float32)
    return torch.ldexp(q, k).flatten(-2)


def _swiglu(gu):
    g, u = gu.clamp(-LIMIT, LIMIT).chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _plain_layer(st):
    c = st["case"]
    T, k, E = c["T"], c["topk"], c["E"]
    if c["hashed"]:
        idx = st["tid2eid"][st["token_ids"].long()].long()
    else:
        idx = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :k]
    z = st["logits"].gather(1, idx)
    s = torch.sqrt(torch.where(z > 20, z, torch.log1p(torch.exp(z.clamp(max=20)))))
    w = ROUTE_SCALE * (s / s.sum(1, keepdim=True) if c["norm"] else s)
    xq = _quantise(st["x"].float())
    e = idx.reshape(-1)                                        # pair p = t * k + j
    xp = xq.repeat_interleave(k, 0).unsqueeze(-1)
    gu = torch.bmm(_mx_dequant(st["w13"][e], st["w13_scale"][e]), xp).squeeze(-1)
    h = _quantise(_swiglu(gu)).unsqueeze(-1)
    o = torch.bmm(_mx_dequant(st["w2"][e], st["w2_scale"][e]), h).view(T, k, -1)
    y = (o * w.unsqueeze(-1)).sum(1)
    if c["shared"]:
        hs = _quantise(_swiglu(xq @ _mx_dequant(st["w13"][E], st["w13_scale"][E]).t()))
        y = y + hs @ _mx_dequant(st["w2"][E], st["w2_scale"][E]).t()
    return {"y": y.to(torch.bfloat16), "idx": idx.to(torch.int32), "w": w}


def _plain_matvec(st):
    c = st["case"]
    if c["fmt"] == "int4":
        q = _nibbles(st["w"])
        q = (q - 16 * (q >= 8)).float()
        w = (q.unflatten(-1, (-1, 128)) * st["scale"].unsqueeze(-1)).flatten(-2)
    elif c["fmt"] == "nvfp4":
        s = st["scale"].view(torch.float8_e4m3fn).float() * st["global"]
        w = (_fp4(st["w"]).unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)
    else:
        w = _mx_dequant(st["w"], st["scale"])
    return (st["x"].float() @ w.t()).to(st["out"].dtype)


def run(st):
    c = st["case"]
    if not own:
        return _plain_layer(st) if c["op"] == "layer" else _plain_matvec(st)
    from fp8_block_scaled_pow2_b200 import moe
    if c["op"] == "layer":
        moe.moe_layer_few_mxfp4(st["x"], st["logits"], st["w13_p"], st["w2_p"], c["I"], st["idx"], st["w"], st["y"],
                                st["workspace"], ROUTE_SCALE, LIMIT, int(c["shared"]), int(c["norm"]),
                                token_ids=st.get("token_ids"), tid2eid=st.get("tid2eid"))
        return {"y": st["y"], "idx": st["idx"], "w": st["w"]}
    if c["fmt"] == "int4":
        moe.moe_matvec_int4g128(st["x"], st["w"], st["scale"], st["out"])
    elif c["fmt"] == "nvfp4":
        moe.moe_matvec_nvfp4(st["x"], st["w"], st["scale"], st["global"], st["out"])
    else:
        moe.moe_matvec_mxfp4(st["x"], st["w"], st["scale"], st["out"])
    return st["out"]


# ------------------------- the definition in 64 bits ------------------------
def _exact_codes(packed):
    out = torch.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=torch.float64, device=packed.device)
    out[..., 0::2] = (packed.to(torch.int16) % 16).double()
    out[..., 1::2] = torch.div(packed.view(torch.uint8).to(torch.int16), 16, rounding_mode="floor").double()
    return out


def _exact_e2m1(packed):
    c = _exact_codes(packed)
    m = c % 8                                     # exponent field floor(m / 2), mantissa bit m % 2
    e, f = torch.floor(m / 2), m % 2
    v = torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e - 1))
    return torch.where(c >= 8, -v, v)


def _exact_e4m3(v):
    """Nearest E4M3 value, ties to even, in float64 (|v| <= 448)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_quantise(x):
    g = x.reshape(*x.shape[:-1], -1, 128)
    r = g.abs().amax(-1, keepdim=True) / 448
    k = torch.ceil(torch.log2(torch.where(r > 0, r, torch.ones_like(r))))
    k = torch.where(torch.exp2(k - 1) >= r, k - 1, k)      # the logarithm may round across a power of two
    k = torch.where(torch.exp2(k) < r, k + 1, k)
    k = torch.where(r > 0, k, torch.zeros_like(k))
    return (_exact_e4m3(g / torch.exp2(k)) * torch.exp2(k)).reshape(x.shape)


def _exact_expert(st, e, rows):
    def weight(name):
        s = torch.exp2(st[name + "_scale"][e].double() - 127).repeat_interleave(32, -1)
        return _exact_e2m1(st[name][e]) * s
    gu = rows @ weight("w13").t()
    I = gu.shape[1] // 2
    g, u = gu[:, :I].clamp(-LIMIT, LIMIT), gu[:, I:].clamp(-LIMIT, LIMIT)
    return _exact_quantise(g * torch.sigmoid(g) * u) @ weight("w2").t()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "matvec":
        x, N, K = st["x"].double(), case["N"], case["K"]
        y = torch.empty((case["M"], N), dtype=torch.float64, device="cuda")
        rows = max(1, 67_108_864 // K)
        for r in range(0, N, rows):
            w, s = st["w"][r:r + rows], st["scale"][r:r + rows]
            if case["fmt"] == "int4":
                v = _exact_codes(w.view(torch.uint8))
                v = torch.where(v > 7, v - 16, v) * s.double().repeat_interleave(128, -1)
            elif case["fmt"] == "nvfp4":
                b = s.to(torch.int32)
                e, f = (b >> 3) & 15, (b & 7).double()
                v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7))
                v = _exact_e2m1(w) * v.repeat_interleave(16, -1) * st["global"].double()
            else:
                v = _exact_e2m1(w) * torch.exp2(s.double() - 127).repeat_interleave(32, -1)
            y[:, r:r + rows] = x @ v.t()
        return y
    T, k = case["T"], case["topk"]
    z = st["logits"].double()
    if case["hashed"]:
        idx = [[int(v) for v in st["tid2eid"][int(t)]] for t in st["token_ids"].tolist()]
    else:
        idx = [sorted(range(case["E"]), key=lambda e, row=row: (-row[e], e))[:k] for row in z.tolist()]
    ids = torch.tensor(idx, device="cuda")
    s = torch.sqrt(torch.logaddexp(torch.zeros_like(z), z)).gather(1, ids)
    w = ROUTE_SCALE * (s / s.sum(1, keepdim=True) if case["norm"] else s)
    xq = _exact_quantise(st["x"].double())
    y = torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
    for e in sorted({e for row in idx for e in row}):
        t, j = (ids == e).nonzero(as_tuple=True)
        y.index_add_(0, t, w[t, j].unsqueeze(1) * _exact_expert(st, e, xq[t]))
    if case["shared"]:
        y += _exact_expert(st, case["E"], xq)
    return {"y": y, "idx": ids.to(torch.int32), "w": w}
