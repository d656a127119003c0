"""The serving operators around the codebook MoE layer, as a model calls them:

- ``norm``: RMS norm before a block, rotated and quantised for the block's GEMMs;
- ``post``: the block's expert rows combined, normed, gated and added to the residual
  stream, with the next block's norm and codes from the same pass;
- ``moe``: the whole MoE layer for the few tokens of a decode batch;
- ``adapter``: a shared codebook projection with low-rank adapters of many requests.

``run`` computes each in a plain form of elementary torch operations, or, where ``own`` is
true, through the package's calls.  Sums and products of values that are quantised later
are taken in 64 bits in the plain form, as a code next to a rounding border would
otherwise depend on the order of a sum.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's input norm: latency alone counts
        dict(name="norm_1x2048", op="norm", T=1, H=2048, act_bits=8),
        # the input norm of a prefill batch
        dict(name="norm_4096x2048", op="norm", T=4096, H=2048, act_bits=8),
        # one token's block output (already combined), sandwich norm, per-channel gate
        dict(name="post_1x2048", op="post", T=1, H=2048, topk=0, shared=1, bf16=True, post_norm=True,
             gate="channel", act_bits=8),
        # a prefill batch's expert rows (top-6 and 2 shared), sandwich norm, per-token gates
        dict(name="post_4096x2048_top6s2", op="post", T=4096, H=2048, topk=6, shared=2, bf16=False,
             post_norm=True, gate="token", act_bits=8),
        # batch-1 decode of a 128-expert layer: 8 experts' weights, latency-bound
        dict(name="moe_1x128e", op="moe", T=1, E=128, topk=8, shared=0, H=2048, F=768, bits_gu=4, bits_d=4,
             act_bits=4, renorm=True),
        # a small decode batch with shared experts and mixed 3- and 2-bit codebooks
        dict(name="moe_8x64e2s", op="moe", T=8, E=64, topk=6, shared=2, H=2048, F=1408, bits_gu=3, bits_d=2,
             act_bits=4, renorm=True),
        # the largest decode batch: most of the 128 experts take part, HBM-bound
        dict(name="moe_32x128e", op="moe", T=32, E=128, topk=8, shared=0, H=2048, F=768, bits_gu=4, bits_d=4,
             act_bits=4, renorm=True),
        # few wide experts, 8-bit activations
        dict(name="moe_16x8e", op="moe", T=16, E=8, topk=2, shared=0, H=4096, F=14336, bits_gu=4, bits_d=4,
             act_bits=8, renorm=True),
        # one request with its adapter beside the projection
        dict(name="adapter_1x2560x9728", op="adapter", T=1, K=2560, N=9728, bits=4, act_bits=8, rank=16,
             adapters=8, order="tokens"),
        # a decode batch, nearly every request with another adapter, some with none
        dict(name="adapter_16x9728x2560", op="adapter", T=16, K=9728, N=2560, bits=4, act_bits=4, rank=32,
             adapters=16, order="tokens"),
        # the prompts of a few short requests, ragged
        dict(name="adapter_333x2560x9728", op="adapter", T=333, K=2560, N=9728, bits=4, act_bits=8, rank=64,
             adapters=8, order="requests"),
        # a full prefill batch of several requests
        dict(name="adapter_4096x2560x9728", op="adapter", T=4096, K=2560, N=9728, bits=4, act_bits=4, rank=16,
             adapters=8, order="requests"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "post", "moe", "adapter"])
    act_bits = rng.choice([4, 8])
    if op == "norm":
        return dict(op=op, T=_log_int(rng, 1, 4096), H=32 * rng.randint(16, 128), act_bits=act_bits)
    if op == "post":
        topk = rng.choice([0, 1, 2, 4, 6, 8])
        return dict(op=op, T=_log_int(rng, 1, 2048), H=32 * rng.randint(16, 128), topk=topk,
                    shared=rng.randint(0, 2) if topk else 1, bf16=rng.random() < 0.5,
                    post_norm=rng.random() < 0.75, gate=rng.choice(["none", "channel", "token"]),
                    act_bits=act_bits)
    if op == "moe":
        E = rng.choice([8, 16, 40, 64, 100, 128])
        return dict(op=op, T=_log_int(rng, 1, 32), E=E, topk=rng.randint(1, min(E, 8)), shared=rng.randint(0, 2),
                    H=32 * rng.randint(16, 80), F=32 * rng.randint(12, 48), bits_gu=rng.randint(2, 4),
                    bits_d=rng.randint(2, 4), act_bits=act_bits, renorm=rng.random() < 0.75)
    T = _log_int(rng, 1, 4096)
    return dict(op=op, T=T, K=32 * rng.randint(16, 80), N=16 * rng.randint(32, 608), bits=rng.randint(2, 4),
                act_bits=act_bits, rank=8 * rng.randint(1, 8), adapters=_log_int(rng, 1, 32),
                order=rng.choice(["tokens", "requests"]))


# ------------------------------------------------------------------ inputs
def _act(gen, T, K):
    """Layer activations in bf16: normal, with two outlier channels."""
    x = torch.randn((T, K), generator=gen, device=DEV)
    x[:, 3] *= 40
    x[:, 77 % K] *= 40
    return x.to(torch.bfloat16)


def _codes(gen, T, K, act_bits):
    """Quantised activations as the packed codes and scales of an earlier call."""
    q_max = 7 if act_bits == 4 else 127
    v = torch.randn((T, K), generator=gen, device=DEV)
    m = v.abs().amax(1, keepdim=True)
    q = torch.round(v / m * q_max).to(torch.int32)
    scales = (m[:, 0] / q_max).contiguous()
    if act_bits == 8:
        return q.to(torch.int8).view(torch.uint8), scales
    return ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8), scales


def _weights(gen, E, N, K, bits):
    """Packed indices [E][N][K*bits/8] (LSB-first) and fp16 codebooks [E][N][2^bits]."""
    idx = torch.randint(0, 256, (E, N, K * bits // 8), generator=gen, device=DEV, dtype=torch.uint8)
    cb = torch.randn((E, N, 1 << bits), generator=gen, device=DEV) * 0.02
    cb = cb.sort(dim=-1).values
    cb[..., -1] = 0.08
    return dict(idx=idx, cb=cb.to(torch.float16), K=K, bits=bits)


def _block(K):
    return K & -K


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    s = dict(c)
    if c["op"] in ("norm", "post"):
        T, H = c["T"], c["H"]
        s["x"] = _act(gen, T, H)                      # the residual stream
        s["w"] = 1 + 0.1 * rand(H)
        s["had"] = _hadamard(_block(H))
        if c["op"] == "post":
            k, n_sh = c["topk"], c["shared"]
            rows = T * k + n_sh * T
            s["rows"] = (0.3 * rand(rows, H)).to(torch.bfloat16 if c["bf16"] else torch.float32)
            s["slots"] = s["tw"] = None
            if k:
                s["slots"] = torch.randperm(T * k, generator=gen, device=DEV).view(T, k).to(torch.int32)
                s["tw"] = torch.softmax(rand(T, k), 1)
            s["pw"] = 1 + 0.1 * rand(H) if c["post_norm"] else None
            s["g"] = None
            if c["gate"] != "none":
                s["g"] = (0.5 + 0.2 * rand(1 if c["gate"] == "channel" else T, H)).to(torch.bfloat16)
        return s
    if c["op"] == "moe":
        T, n = c["T"], c["E"] + c["shared"]
        s["codes"], s["scales"] = _codes(gen, T, c["H"], c["act_bits"])
        s["logits"] = rand(T, c["E"])
        s["had"] = _hadamard(_block(c["F"]))
        mats = dict(gate=(c["F"], c["H"], c["bits_gu"]), up=(c["F"], c["H"], c["bits_gu"]),
                    down=(c["H"], c["F"], c["bits_d"]))
        for name, (N, K, bits) in mats.items():
            s[name] = _weights(gen, n, N, K, bits)
    else:
        T, K, N, R, A = c["T"], c["K"], c["N"], c["rank"], c["adapters"]
        s["codes"], s["scales"] = _codes(gen, T, K, c["act_bits"])
        s["x"] = _act(gen, T, K)
        s["wt"] = _weights(gen, 1, N, K, c["bits"])
        s["a"] = (rand(A, R, K) / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (0.1 * rand(A, N, R)).to(torch.bfloat16)
        s["as"] = 0.5 + torch.rand(A, generator=gen, device=DEV)
        of = torch.randint(-1, A, (T,), generator=gen, device=DEV, dtype=torch.int32)
        if c["order"] == "requests":                  # runs of tokens, in the requests' order
            cut = torch.sort(torch.randint(0, T, (A,), generator=gen, device=DEV)).values
            req = torch.searchsorted(cut, torch.arange(T, device=DEV), right=True)
            ids = torch.cat([torch.randperm(A, generator=gen, device=DEV), torch.tensor([-1], device=DEV)])
            of = ids[req].to(torch.int32)
        if T == 1:
            of = of.clamp(min=0)
        s["of"] = of
    if own:                                           # the weights' layout that a server makes once
        import codebook_bit_quantized_amd as cbq
        for name in ("gate", "up", "down", "wt"):
            if name in s:
                w = s[name]
                s[name + "_own"] = cbq.prepack_weights(cbq.CodebookWeights(idx=w["idx"], codebook=w["cb"], K=w["K"],
                                                                           bits=w["bits"]))
        if c["op"] == "moe":
            n_ws = cbq.moe_few_workspace(c["T"], c["topk"], c["shared"], c["H"], c["F"], c["act_bits"])
        else:
            n_ws = cbq.adapter_workspace(c["T"], c["rank"])
        s["ws"] = torch.empty((n_ws,), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _hadamard(b):
    i = torch.arange(b, device=DEV)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 8)
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).double()


def _rotate_quantise(v, had, act_bits):
    """Block Hadamard transform and per-row absmax codes: (codes as fp32, scales)."""
    b = had.shape[0]
    u = (v.double().reshape(-1, b) @ had).reshape(v.shape).float()
    q_max = 7.0 if act_bits == 4 else 127.0
    m = u.abs().amax(1, keepdim=True)
    s = (m.double() / q_max).float()
    r = (u.double() / torch.where(s > 0, s, 1).double()).float()
    q = torch.round(r).clamp(-8.0 if act_bits == 4 else -127.0, q_max)
    return q, (s * torch.tensor(1 / math.sqrt(b), device=DEV, dtype=torch.float32))[:, 0]


def _rms_norm(v64, w):
    return v64 * torch.rsqrt(v64.square().mean(1, keepdim=True) + EPS) * w.double()


def _bf16(v64):
    return v64.float().to(torch.bfloat16)


def _norm_outputs(v, w, had, act_bits):
    normed = _bf16(_rms_norm(v.double(), w))
    q, scales = _rotate_quantise(normed, had, act_bits)
    return _code_values(q, scales, act_bits, normed)


def _code_values(q, scales, act_bits, normed):
    """What the codes stand for; 4-bit ones as the even and the odd channels."""
    if act_bits == 8:
        return dict(normed=normed, scales=scales, values=q * scales[:, None])
    return dict(normed=normed, scales=scales, even=q[:, 0::2] * scales[:, None], odd=q[:, 1::2] * scales[:, None])


def _unpack_codes(codes, act_bits):
    if act_bits == 8:
        return codes.view(torch.int8).float()
    c = codes.view(torch.int8)
    return torch.stack(((c << 4) >> 4, c >> 4), -1).flatten(-2).float()


def _indices(idx, bits):
    if bits == 3:
        b = idx.reshape(*idx.shape[:-1], -1, 3).int()
        v = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        sh = torch.arange(0, 24, 3, device=DEV)
    else:
        v = idx.int()
        sh = torch.arange(0, 8, bits, device=DEV)
    return ((v[..., None] >> sh) & ((1 << bits) - 1)).flatten(-2)


def _dense(w, sel, dtype):
    """Weights [len(sel)][N][K] of the selected experts."""
    idx, cb = (w["idx"], w["cb"]) if sel is None else (w["idx"][sel], w["cb"][sel])
    return cb.to(dtype).gather(-1, _indices(idx, w["bits"]).long())


def _plain_post(s):
    T = s["T"]
    rows = s["rows"].double()
    k, n_sh = s["topk"], s["shared"]
    y = rows[T * k:].view(n_sh, T, -1).sum(0)
    if k:
        y = y + (rows[s["slots"].long()] * s["tw"].double()[..., None]).sum(1)
    if s["pw"] is not None:
        y = _rms_norm(y, s["pw"])
    if s["g"] is not None:
        y = y * s["g"].double()
    out = _bf16(s["x"].double() + 0.5 * y)
    return dict(out=out, **_norm_outputs(out, s["w"], s["had"], s["act_bits"]))


def _plain_moe(s):
    T, E, k, n_sh = s["T"], s["E"], s["topk"], s["shared"]
    top, ids = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    p = torch.exp(top - top[:, :1])
    wts = p[:, :k] / (p[:, :k] if s["renorm"] else p).sum(1, keepdim=True)
    ids = ids[:, :k]
    if T * k < E:                                     # the chosen experts, one entry per choice
        sel = ids.flatten()
        c = wts.flatten()[:, None] * (torch.arange(T * k, device=DEV)[:, None] // k == torch.arange(T, device=DEV))
    else:                                             # all experts
        sel = torch.arange(E, device=DEV)
        c = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter(1, ids, wts).T
    sel = torch.cat([sel, torch.arange(E, E + n_sh, device=DEV)])
    c = torch.cat([c, torch.ones((n_sh, T), dtype=torch.float64, device=DEV)])
    x = _unpack_codes(s["codes"], s["act_bits"]).double() * s["scales"].double()[:, None]

    def project(w):
        W = _dense(w, sel, torch.float64)
        return (W.reshape(-1, W.shape[2]) @ x.T).view(W.shape[0], W.shape[1], T).transpose(1, 2)

    g, u = project(s["gate"]), project(s["up"])
    h = (g * torch.sigmoid(g) * u).reshape(-1, s["F"])
    q, scales = _rotate_quantise(h, s["had"], s["act_bits"])
    h = (q.double() * scales.double()[:, None]).view(len(sel), T, s["F"])
    out = torch.bmm(h, _dense(s["down"], sel, torch.float64).transpose(1, 2).contiguous())
    return _bf16((out * c[..., None]).sum(0))


def _plain_adapter(s):
    T, A, R = s["T"], s["adapters"], s["rank"]
    W = _dense(s["wt"], None, torch.float32)[0]
    base = (_unpack_codes(s["codes"], s["act_bits"]) @ W.T) * s["scales"][:, None]
    t = (s["x"].float() @ s["a"].float().view(A * R, -1).T).view(T, A, R) * s["as"][:, None]
    mine = s["of"].long()[:, None] == torch.arange(A, device=DEV)
    t = torch.where(mine[..., None], t, 0).view(T, A * R)
    return base + t @ s["b"].float().transpose(0, 1).reshape(-1, A * R).T


# ------------------------------------------------------------------ the framework's calls
def _own_code_values(normed, codes, scales, act_bits):
    c = codes.view(torch.int8)
    if act_bits == 8:
        return dict(normed=normed, scales=scales, values=c * scales[:, None])
    return dict(normed=normed, scales=scales, even=((c << 4) >> 4) * scales[:, None], odd=(c >> 4) * scales[:, None])


def _own(s):
    import codebook_bit_quantized_amd as cbq
    ab = s["act_bits"]
    if s["op"] == "norm":
        return _own_code_values(*cbq.norm_rotate_quantize(s["x"], s["w"], EPS, ab), ab)
    if s["op"] == "post":
        out, normed, codes, scales = cbq.combine_norm_residual(
            s["rows"], s["x"], s["slots"], s["tw"], n_shared=s["shared"], post_weight=s["pw"], eps=EPS, gate=s["g"],
            scale=0.5, next_weight=s["w"], act_bits=ab)
        return dict(out=out, **_own_code_values(normed, codes, scales, ab))
    if s["op"] == "moe":
        return cbq.moe_ffn_few(s["codes"], s["scales"], s["logits"], s["gate_own"], s["up_own"], s["down_own"],
                               s["topk"], s["shared"], ab, renormalize=s["renorm"], ws=s["ws"])
    return cbq.codebook_adapter_gemm(s["codes"], s["scales"], ab, s["wt_own"], s["x"], s["a"], s["b"], s["of"],
                                     s["as"], ws=s["ws"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "norm":
        return _norm_outputs(state["x"], state["w"], state["had"], state["act_bits"])
    if op == "post":
        return _plain_post(state)
    if op == "moe":
        return _plain_moe(state)
    return _plain_adapter(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    T, ab = c["T"], c["act_bits"]
    if c["op"] == "norm":
        H = c["H"]
        return dict(bytes=T * H * (2 + 2 + ab / 8) + 4 * H + 4 * T, flops=T * H * (6 + math.log2(_block(H))))
    if c["op"] == "post":
        H, n = c["H"], c["topk"] + c["shared"]
        gate = {"none": 0, "channel": 2 * H, "token": 2 * T * H}[c["gate"]]
        return dict(bytes=T * H * (n * (2 if c["bf16"] else 4) + 2 + 2 + 2 + ab / 8) + gate + 8 * H + 8 * T * n,
                    flops=T * H * (2 * n + 14 + math.log2(_block(H))))
    if c["op"] == "moe":
        E, k, n_sh, H, F = c["E"], c["topk"], c["shared"], c["H"], c["F"]
        active = E * (1 - (1 - k / E) ** T) + n_sh    # expected for independent choices
        mat = lambda N, K, bits: N * K * bits / 8 + N * 2 * 2 ** bits  # noqa: E731
        per = 2 * mat(F, H, c["bits_gu"]) + mat(H, F, c["bits_d"])
        return dict(bytes=active * per + T * (H * ab / 8 + 4 + 4 * E + 2 * H), flops=6 * T * (k + n_sh) * H * F)
    K, N, R = c["K"], c["N"], c["rank"]
    used = c["adapters"] * (1 - (1 - 1 / (c["adapters"] + 1)) ** T)
    return dict(bytes=N * K * c["bits"] / 8 + N * 2 * 2 ** c["bits"] + T * (K * ab / 8 + 2 * K + 8 + 4 * N)
                + used * 2 * R * (K + N), flops=2 * T * N * K + 2 * T * R * (K + N))


# ------------------------------------------------------------------ the definitions in 64 bits
def _butterflies(v, b):
    """The block transform by successive sums and differences."""
    v = v.clone()
    n, K = v.shape
    h = 1
    while h < b:
        w = v.view(n, K // (2 * h), 2, h)
        v = torch.stack((w[:, :, 0] + w[:, :, 1], w[:, :, 0] - w[:, :, 1]), 2).reshape(n, K)
        h *= 2
    return v


def _exact_codes(v64, act_bits):
    K = v64.shape[1]
    b = _block(K)
    u = _butterflies(v64, b).float().double()         # the quantiser works on the transform rounded to fp32
    top = 7 if act_bits == 4 else 127
    s = (u.abs().max(dim=1, keepdim=True).values / top).float().double()
    q = torch.round((u / s.clamp(min=1e-300)).float()).double()
    q = q.clamp(-top - (1 if act_bits == 4 else 0), top)
    return q, s / math.sqrt(b)


def _exact_norm(x64, w, act_bits):
    n = x64 / torch.sqrt((x64 * x64).sum(1, keepdim=True) / x64.shape[1] + EPS) * w.double()
    q, s = _exact_codes(n.float().to(torch.bfloat16).double(), act_bits)
    d = dict(normed=n, scales=s[:, 0])
    if act_bits == 8:
        d["values"] = q * s
    else:
        d["even"], d["odd"] = q[:, ::2] * s, q[:, 1::2] * s
    return d


def _exact_matrix(w, e):
    """W[e] in fp64: bit p of a row's stream is bit p % 8 of byte p // 8."""
    bits, K = w["bits"], w["K"]
    row = w["idx"][e].to(torch.int64)
    a = torch.zeros((row.shape[0], K), dtype=torch.int64, device=DEV)
    for j in range(bits):
        p = torch.arange(K, device=DEV) * bits + j
        a |= ((row[:, p // 8] >> (p % 8)) & 1) << j
    return torch.gather(w["cb"][e].double(), 1, a)


def _exact_tokens(s):
    c = s["codes"].to(torch.int64)
    if s["act_bits"] == 8:
        q = torch.where(c > 127, c - 256, c)
    else:
        q = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.int64, device=DEV)
        q[:, ::2], q[:, 1::2] = c % 16, c // 16
        q = torch.where(q > 7, q - 16, q)
    return q.double() * s["scales"].double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    T, ab = s["T"], s["act_bits"]
    if s["op"] == "norm":
        return _exact_norm(s["x"].double(), s["w"], ab)
    if s["op"] == "post":
        k = s["topk"]
        y = torch.zeros((T, s["H"]), dtype=torch.float64, device=DEV)
        for j in range(k):
            y += s["tw"][:, j:j + 1].double() * s["rows"][s["slots"][:, j].long()].double()
        for j in range(s["shared"]):
            y += s["rows"][T * k + j * T:T * k + (j + 1) * T].double()
        if s["pw"] is not None:
            y = y / torch.sqrt((y * y).sum(1, keepdim=True) / s["H"] + EPS) * s["pw"].double()
        if s["g"] is not None:
            y = y * s["g"].double()
        out = s["x"].double() + y / 2
        return dict(out=out, **_exact_norm(out.float().to(torch.bfloat16).double(), s["w"], ab))
    x = _exact_tokens(s)
    if s["op"] == "adapter":
        out = x @ _exact_matrix(s["wt"], 0).T
        for a in range(s["adapters"]):
            t = torch.nonzero(s["of"] == a)[:, 0]
            d = s["x"][t].double() @ s["a"][a].double().T @ s["b"][a].double().T
            out[t] += s["as"][a].double() * d
        return out
    E, k = s["E"], s["topk"]
    l = s["logits"].double()
    y = torch.zeros((T, s["H"]), dtype=torch.float64, device=DEV)
    before = (l[:, None, :] > l[:, :, None]).sum(2)   # experts ahead of e, then those with its value and a lower id
    tie = (l[:, None, :] == l[:, :, None]) & (torch.arange(E, device=DEV)[None, :] < torch.arange(E, device=DEV)[:, None])
    chosen = before + tie.sum(2) < k
    p = torch.exp(l - l.max(1, keepdim=True).values)
    p = p / (p * chosen if s["renorm"] else p).sum(1, keepdim=True)
    for e in range(E + s["shared"]):
        t = torch.nonzero(chosen[:, e])[:, 0] if e < E else torch.arange(T, device=DEV)
        if len(t) == 0:
            continue
        g, u = x[t] @ _exact_matrix(s["gate"], e).T, x[t] @ _exact_matrix(s["up"], e).T
        q, sc = _exact_codes(g / (1 + torch.exp(-g)) * u, ab)
        o = (q * sc) @ _exact_matrix(s["down"], e).T
        y[t] += o * (p[t, e:e + 1] if e < E else 1)
    return y
