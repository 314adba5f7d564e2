"""The attention side of a block around the MoE layer, as workloads to time and compare.

Three operators that run one after the other in front of the routed-expert
layer when a prompt or a single token goes through a block:

  fp8_linear    y = x W^T with E4M3 weights, one scale per 128 x 128 block of
                W, and x quantised to E4M3 with one scale per token and 128
                columns (the source's dense-weight format);
  qk_norm_rope  RMS norm of every query and key head and the rotary position
                embedding of it, in one pass;
  attention     softmax attention over packed sequences of different lengths,
                causal, with grouped heads: whole prompts, chunks of a prompt
                after a prefix, and single tokens over a long cache.

`run` computes a pass either with the library's operators (own = True) or in
plain torch operations in float32 (own = False); `exact` does it in float64.
"""
import math
import random

import torch

own = False

HIDDEN, INTER = 4096, 2048  # the MoE layer's hidden and intermediate size
FP8_MAX = 448.0             # largest E4M3 value


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through the fused q|k|v projection (32 query, 8 key and 8 value heads of 128): latency
        dict(name="fp8_decode_t1", op="fp8_linear", T=1, N=6144, K=HIDDEN, scale="e8m0"),
        # the 64-token decode batch through the output projection; float32 scales
        dict(name="fp8_decode_t64", op="fp8_linear", T=64, N=HIDDEN, K=HIDDEN, scale="float32"),
        # a ragged batch through a projection whose sizes fill no block (the last blocks of N and K are partial)
        dict(name="fp8_ragged_t509", op="fp8_linear", T=509, N=1000, K=2064, scale="e8m0"),
        # the largest prefill batch through the fused q|k|v projection, in each scale type
        dict(name="fp8_prefill_t16384", op="fp8_linear", T=16384, N=6144, K=HIDDEN, scale="e8m0"),
        dict(name="fp8_prefill_t4096_f32", op="fp8_linear", T=4096, N=HIDDEN, K=HIDDEN, scale="float32"),
        # a 4-token decode step, far into a long context: latency
        dict(name="rope_decode_t4", op="qk_norm_rope", T=4, Hq=32, Hkv=8, D=128, R=128, tail=False, interleaved=False,
             P=131072),
        # a whole prefill batch; and one with a single key head and a partial rotation on the tail of the head
        dict(name="rope_prefill_t16384", op="qk_norm_rope", T=16384, Hq=32, Hkv=8, D=128, R=128, tail=False,
             interleaved=False, P=16384),
        dict(name="rope_partial_t2049", op="qk_norm_rope", T=2049, Hq=64, Hkv=1, D=128, R=64, tail=True,
             interleaved=True, P=8192),
        # a 4-token decode step over short caches: latency; a 64-token one over caches of very different lengths
        dict(name="attn_decode_b4", op="attention", kind="decode", B=4, q=1, kv=1024, Hq=32, Hkv=8, D=128, lens=1),
        dict(name="attn_decode_b64", op="attention", kind="decode", B=64, q=1, kv=8192, Hq=32, Hkv=8, D=128, lens=2),
        # one prompt of 16384 tokens; eleven packed prompts of different lengths, 64-wide heads
        dict(name="attn_prompt_t16384", op="attention", kind="prompt", B=1, q=16384, kv=16384, Hq=32, Hkv=8, D=128,
             lens=3),
        dict(name="attn_packed_t8192", op="attention", kind="prompt", B=11, q=8192, kv=8192, Hq=16, Hkv=16, D=64,
             lens=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8_linear", "qk_norm_rope", "attention", "attention"])
    if op == "fp8_linear":
        while True:
            c = dict(op=op, T=_log(rng, 1, 16384), N=_log(rng, 64, 8192), K=16 * _log(rng, 8, 512),
                     scale=rng.choice(["e8m0", "float32"]))
            if c["T"] * c["N"] * c["K"] <= 16384 * 6144 * HIDDEN:
                return c
    if op == "qk_norm_rope":
        while True:
            D = rng.choice([64, 128, 128, 256])
            Hkv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, T=_log(rng, 1, 32768), Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, D=D,
                     R=rng.choice([D, D // 2]), tail=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                     P=_log(rng, 64, 131072))
            if c["T"] * (c["Hq"] + Hkv) * D <= 16384 * 40 * 128:
                return c
    kind = rng.choice(["decode", "decode", "prompt", "chunk"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    while True:
        if kind == "decode":
            B, q, kv = _log(rng, 1, 128), 1, _log(rng, 1, 131072)
        elif kind == "chunk":
            B, q, kv = _log(rng, 1, 8), _log(rng, 2, 2048), _log(rng, 128, 32768)
        else:
            B, q = _log(rng, 1, 32), _log(rng, 32, 16384)
            kv = q
        c = dict(op=op, kind=kind, B=B, q=q, kv=kv, Hq=Hq, Hkv=Hkv, D=D, lens=rng.randrange(1 << 30))
        if kind == "chunk" and q > kv:
            continue
        rows = kv if kind == "prompt" else B * kv
        if rows * Hkv * D > 64 * 8192 * 8 * 128 or _attn_work(c)["flops"] > 4 * 128 * 32 * 16384 * 8192:
            continue
        return c


def _lengths(case):
    """Query and key length of every sequence of an attention case."""
    r = random.Random(case["lens"])
    B = case["B"]
    if case["kind"] == "decode":      # one token each; the first cache is full, the others anywhere
        return [1] * B, [case["kv"]] + [r.randint(1, case["kv"]) for _ in range(B - 1)]
    if case["kind"] == "chunk":       # a chunk of a prompt after a prefix of any length
        lq = [case["q"]] + [r.randint(1, case["q"]) for _ in range(B - 1)]
        return lq, [case["kv"]] + [r.randint(n, case["kv"]) for n in lq[1:]]
    cuts = sorted(r.randint(0, case["q"]) for _ in range(B - 1))
    if B >= 6:                        # among many prompts one of a single token, and an empty one
        cuts[1] = min(cuts[0] + 1, case["q"])
        cuts[3] = cuts[2] = max(cuts[1], cuts[2])
        cuts.sort()
    cuts = [0] + cuts + [case["q"]]
    lq = [b - a for a, b in zip(cuts, cuts[1:])]
    return lq, list(lq)


# ------------------------------------------------------------------ the least work
def work(case):
    if case["op"] == "fp8_linear":
        T, N, K = case["T"], case["N"], case["K"]
        blocks = -(-N // 128) * -(-K // 128)
        return dict(bytes=2 * T * K + N * K + blocks * (1 if case["scale"] == "e8m0" else 4) + 2 * T * N,
                    flops=2 * T * N * K)
    if case["op"] == "qk_norm_rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return dict(bytes=4 * n + 4 * min(case["T"], case["P"]) * case["R"] + 4 * case["T"] + 8 * case["D"],
                    flops=6 * n)
    return _attn_work(case)


def _attn_work(case):
    lq, lk = _lengths(case)
    # query i of a sequence sees keys 0 .. lk - lq + i
    seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
    rows = sum(lq)
    return dict(bytes=2 * case["D"] * (2 * rows * case["Hq"] + 2 * sum(lk) * case["Hkv"]) + 12 * case["B"],
                flops=4 * case["D"] * case["Hq"] * seen)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) * std)

    st = dict(case=case)
    if case["op"] == "fp8_linear":
        T, N, K = case["T"], case["N"], case["K"]
        x = normal(T, K)
        hot = torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")
        x[:, hot] *= 20  # a few outlier channels, as activations have
        w, s = _quantise_weight(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K), case["scale"])
        st.update(x=x, w=w, s=s)
    elif case["op"] == "qk_norm_rope":
        T, Hq, Hkv, D, R = (case[k] for k in ("T", "Hq", "Hkv", "D", "R"))
        qkv = normal(T, (Hq + 2 * Hkv) * D, std=3.0)
        pos = torch.randint(0, case["P"], (T,), generator=g, device="cuda", dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        ang = torch.arange(case["P"], dtype=torch.float64, device="cuda")[:, None] * inv
        st.update(q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D), pos=pos,
                  qw=1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
                  kw=1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
                  cs=torch.cat([ang.cos(), ang.sin()], 1).float(),
                  q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
                  k_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda"))
    else:
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lq, lk = _lengths(case)
        T = sum(lq)
        if case["kind"] == "prompt":  # q, k and v side by side in the projection's output
            qkv = normal(T, (Hq + 2 * Hkv) * D)
            qkv[:, :Hq * D] *= 2
            q, k, v = (qkv[:, a * D:(a + h) * D].view(T, h, D) for a, h in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
            start = None
        else:                         # a cache with room for kv tokens of every sequence
            q = normal(T, Hq, D, std=2.0)
            k, v = normal(case["B"] * case["kv"], Hkv, D), normal(case["B"] * case["kv"], Hkv, D)
            start = [b * case["kv"] for b in range(case["B"])]

        def ints(a):
            return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")

        cu = [0]
        for n in lq:
            cu.append(cu[-1] + n)
        st.update(q=q, k=k, v=v, lq=lq, lk=lk, cu=ints(cu), start=ints(start), len=ints(lk if start else None), q0=cu,
                  k0=start or cu, most=(max(lq), max(lk)),
                  out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"))
    if own:
        from mxfp4_routed_expert_moe_amd import attention as A
        if case["op"] == "fp8_linear":
            st["y"] = torch.empty(case["T"], case["N"], dtype=torch.bfloat16, device="cuda")
            st["ws"] = A.fp8_linear_workspace(case["T"], case["N"], case["K"])
        elif case["op"] == "attention":
            st["ws"] = A.attention_workspace(st["q"], st["k"], case["B"], *st["most"])
    return st


def _quantise_weight(w, kind):
    """[N, K] float32 -> E4M3 codes [N, K] and one scale per 128 x 128 block: E8M0 bytes or float32."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.zeros(nb * 128, kb * 128, device=w.device)
    p[:N, :K] = w
    p = p.view(nb, 128, kb, 128)
    s = p.abs().amax((1, 3)).clamp_min(1e-20) / FP8_MAX
    if kind == "e8m0":
        e = torch.ceil(torch.log2(s))
        s, kept = torch.exp2(e), (e + 127).to(torch.uint8)
    else:
        kept = s
    codes = (p / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)
    return codes[:N, :K].contiguous(), kept


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if not own:
        return {"fp8_linear": _plain_linear, "qk_norm_rope": _plain_rope, "attention": _plain_attention}[case["op"]](st)
    from mxfp4_routed_expert_moe_amd import attention as A
    if case["op"] == "fp8_linear":
        return A.fp8_linear(st["x"], st["w"], st["s"], y=st["y"], ws=st["ws"])
    if case["op"] == "qk_norm_rope":
        return A.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["pos"], st["cs"],
                              rot_offset=case["D"] - case["R"] if case["tail"] else 0,
                              interleaved=case["interleaved"], q_out=st["q_out"], k_out=st["k_out"])
    return A.attention(st["q"], st["k"], st["v"], st["cu"], st["most"][0], kv_start=st["start"], kv_len=st["len"],
                       max_kv=st["most"][1], out=st["out"], ws=st["ws"])


def _power(e):
    """2^e in float32 for int32 e in -126 .. 127."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_linear(st):
    x, w, s = st["x"].float(), st["w"].float(), st["s"]
    T, K = x.shape
    N = w.shape[0]
    kb = -(-K // 128)
    xp = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(T, kb, 128)
    amax = xp.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    if st["case"]["scale"] == "e8m0":  # the least power of two with amax / scale <= 448; both divisions are exact
        m, e = torch.frexp(amax)      # amax = m 2^e, 0.5 <= m < 1
        sx = _power(e - 9 + (m > 0.875).int())
        codes = (xp / sx).to(torch.float8_e4m3fn)
        s = _power(s.int() - 127)
    else:
        top = torch.full_like(amax, FP8_MAX)  # a tensor: torch multiplies by the reciprocal of a number
        sx = amax / top
        codes = (xp * (top / amax)).to(torch.float8_e4m3fn)
    xq = (codes.float() * sx).view(T, kb * 128)[:, :K]
    wq = w * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return (xq @ wq.t()).bfloat16()


def _rotate(x, cs, R, off, interleaved):
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    r = x[..., off:off + R]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    ra, rb = a * c - b * s, b * c + a * s
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([x[..., :off], r, x[..., off + R:]], -1)


def _rope_any(st, dtype):
    case = st["case"]
    cs = st["cs"][st["pos"].long()].to(dtype)
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.to(dtype)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(dtype)
        out.append(_rotate(x, cs, case["R"], case["D"] - case["R"] if case["tail"] else 0, case["interleaved"]))
    return out


def _plain_rope(st):
    return tuple(x.bfloat16() for x in _rope_any(st, torch.float32))


def _plain_attention(st):
    case = st["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    out = st["out"]
    for a, n, k0, m in zip(st["q0"], st["lq"], st["k0"], st["lk"]):
        if n == 0:
            continue
        k = st["k"][k0:k0 + m].float().permute(1, 2, 0).contiguous()  # [Hkv, D, m]
        v = st["v"][k0:k0 + m].float().transpose(0, 1).contiguous()   # [Hkv, m, D]
        step = max(1, (1 << 28) // (Hq * m))                          # at most 1 GiB of scores at a time
        for i in range(0, n, step):
            r = min(step, n - i)
            q = st["q"][a + i:a + i + r].float().view(r, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * r, D)
            z = torch.matmul(q, k).view(Hkv, G, r, m) * (1 / math.sqrt(D))
            if n > 1:
                seen = torch.arange(m, device="cuda") <= torch.arange(i, i + r, device="cuda")[:, None] + (m - n)
                z = z.masked_fill(~seen, float("-inf"))
            p = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(p.view(Hkv, G * r, m), v).view(Hkv, G, r, D) / p.sum(-1, keepdim=True)
            out[a + i:a + i + r] = o.permute(2, 0, 1, 3).reshape(r, Hq, D).bfloat16()
    return out


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "attention" and _attn_work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "fp8_linear":
        return _exact_linear(st)
    if case["op"] == "qk_norm_rope":
        return _exact_rope(st)
    return _exact_attention(st)


def _exact_linear(st):
    # The quantiser is defined in float32 (E8M0: the division is exact; float32 scales: the code is that of the
    # float32 product of x and the float32 quotient 448 / amax); the sums of the products are in 64 bits.
    x = st["x"].double()
    w = st["w"].double()
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    floor = 2.0 ** -100
    for b in range(0, x.shape[1], 128):
        xb = x[:, b:b + 128]
        top = torch.maximum(xb.abs().max(1).values, torch.tensor(floor, dtype=torch.float64, device="cuda"))
        sw = st["s"][:, b // 128]
        if st["case"]["scale"] == "e8m0":
            sx = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), torch.ceil(torch.log2(top / 448)))
            sx = torch.where(top / sx > 448, 2 * sx, sx)          # where log2 rounded
            sx = torch.where(top / sx <= 224, sx / 2, sx)
            code = (xb / sx[:, None]).float().to(torch.float8_e4m3fn).double()
            sw = torch.pow(2.0, sw.double() - 127)
        else:
            sx = (top / 448).float().double()
            inv = (448 / top).float().double()
            code = (xb * inv[:, None]).float().to(torch.float8_e4m3fn).double()
            sw = sw.double()
        part = torch.matmul(code, w[:, b:b + 128].t().contiguous())
        y += part * sx[:, None] * torch.repeat_interleave(sw, 128)[:w.shape[0]]
    return y


def _exact_rope(st):
    case = st["case"]
    R = case["R"]
    off = case["D"] - R if case["tail"] else 0
    res = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.double()
        n = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6) * w.double()
        y = n.clone()
        half = torch.arange(R // 2, device="cuda")
        i, j = (off + 2 * half, off + 2 * half + 1) if case["interleaved"] else (off + half, off + half + R // 2)
        t = st["cs"].double()[st["pos"].long()].unsqueeze(1)
        z = torch.complex(n[..., i], n[..., j]) * torch.complex(t[..., :R // 2], t[..., R // 2:])
        y[..., i], y[..., j] = z.real, z.imag
        res.append(y)
    return tuple(res)


def _exact_attention(st):
    case = st["case"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for a, n, k0, m in zip(st["q0"], st["lq"], st["k0"], st["lk"]):
        if n == 0:
            continue
        hidden = None
        if n > 1:
            hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(case["Hkv"]):
            k = st["k"][k0:k0 + m, h].double().t().contiguous()
            v = st["v"][k0:k0 + m, h].double()
            for j in range(h * G, h * G + G):
                z = (st["q"][a:a + n, j].double() @ k) / math.sqrt(case["D"])
                if hidden is not None:
                    z.masked_fill_(hidden, float("-inf"))
                out[a:a + n, j] = torch.softmax(z, -1) @ v
    return out
