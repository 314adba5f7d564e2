"""A key/value cache in pages, as workloads to time and compare.

What serving adds to the attention half of a block: sequences whose cached keys
and values lie in pages of one pool, named by a page table.

  paged_append      new keys normed and rotated on their way into the pages,
                    values beside them, the queries of the same tokens normed
                    and rotated too, and per page and head the smallest and the
                    largest key element in each column;
  paged_attention   causal softmax attention over the pages, where groups of
                    sequences hold the same prefix in the same pages;
  select_blocks     for every token and key head the pages whose bounds promise
                    the largest products with its queries;
  sparse_attention  softmax attention over the selected pages alone.

`run` computes a pass either with the library's operators (own = True) or in
plain torch operations in float32 (own = False; the scores that pages are
selected by in float64); `exact` does it in float64.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a 4-token decode step: latency
        dict(name="append_decode_t4", op="paged_append", kind="decode", B=4, q=1, kv=4096, Hq=32, Hkv=8, D=128, page=64,
             R=128, tail=False, interleaved=False, norm=True, lens=1),
        # chunks of seven prompts, which begin and end inside small pages; a partial rotation and no norm
        dict(name="append_ragged_t2049", op="paged_append", kind="chunk", B=7, q=2049, kv=4096, Hq=16, Hkv=4, D=64,
             page=16, R=32, tail=True, interleaved=True, norm=False, lens=2),
        # a whole prefill batch of three prompts
        dict(name="append_prefill_t16384", op="paged_append", kind="prompt", B=3, q=16384, kv=16384, Hq=32, Hkv=8, D=128,
             page=64, R=128, tail=False, interleaved=False, norm=True, lens=3),
        # four samples of one short prompt: latency
        dict(name="prefix_decode_b4", op="paged_attention", kind="decode", B=4, q=1, groups=1, prefix=1024, kv=256,
             Hq=32, Hkv=8, D=128, page=64, lens=4),
        # 64 requests behind one long system prompt, each with a conversation of its own
        dict(name="prefix_decode_b64", op="paged_attention", kind="decode", B=64, q=1, groups=1, prefix=16384, kv=2048,
             Hq=32, Hkv=8, D=128, page=64, lens=5),
        # seven prompts of different lengths, sampled between one and many times; small pages, 64-wide heads
        dict(name="prefix_groups_b96", op="paged_attention", kind="decode", B=96, q=1, groups=7, prefix=4001, kv=1000,
             Hq=16, Hkv=4, D=64, page=16, lens=6),
        # eight questions of a few hundred tokens about one document
        dict(name="prefix_chunk_b8", op="paged_attention", kind="chunk", B=8, q=256, groups=1, prefix=16384, kv=512,
             Hq=32, Hkv=8, D=128, page=64, lens=7),
        # the 64-token decode batch over long contexts
        dict(name="select_decode_b64", op="select_blocks", kind="decode", B=64, q=1, kv=32768, Hq=32, Hkv=8, D=128,
             page=64, k=32, lens=8),
        # a chunk of a prompt far into a long context
        dict(name="select_chunk_t1021", op="select_blocks", kind="chunk", B=1, q=1021, kv=65536, Hq=16, Hkv=2, D=128,
             page=64, k=48, lens=9),
        # four tokens over ordinary contexts: latency
        dict(name="sparse_decode_b4", op="sparse_attention", kind="decode", B=4, q=1, kv=8192, Hq=32, Hkv=8, D=128,
             page=64, k=16, lens=10),
        # a decode batch over long contexts
        dict(name="sparse_decode_b32", op="sparse_attention", kind="decode", B=32, q=1, kv=32768, Hq=32, Hkv=8, D=128,
             page=64, k=64, lens=11),
        # chunks of two prompts over long contexts: neighbouring tokens select much the same pages
        dict(name="sparse_chunk_t509", op="sparse_attention", kind="chunk", B=2, q=509, kv=30000, Hq=32, Hkv=4, D=128,
             page=32, k=40, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged_append", "paged_attention", "paged_attention", "select_blocks", "sparse_attention"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    base = dict(op=op, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 16]), Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 64, 128]),
                lens=rng.randrange(1 << 30))
    while True:
        if op == "paged_append":
            kind = rng.choice(["decode", "chunk", "prompt"])
            B = _log(rng, 1, 128 if kind == "decode" else 16)
            q = 1 if kind == "decode" else _log(rng, 32, 16384)
            kv = q if kind == "prompt" else _log(rng, max(q, 64), 8192 if q <= 8192 else 16384)
            c = dict(base, kind=kind, B=B, q=q, kv=kv, R=rng.choice([D, D // 2]), tail=rng.random() < 0.5,
                     interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
            rows = _rows(c)
            if sum(rows[0]) * (c["Hq"] + 2 * Hkv) * D <= 16384 * 48 * 128 and sum(rows[1]) * Hkv * D <= 1 << 26:
                return c
        elif op == "paged_attention":
            kind = rng.choice(["decode", "decode", "decode", "chunk"])
            B = _log(rng, 1, 128 if kind == "decode" else 12)
            c = dict(base, kind=kind, B=B, q=1 if kind == "decode" else _log(rng, 2, 512), groups=_log(rng, 1, B),
                     prefix=rng.choice([0, 1, 1, 1]) and _log(rng, 16, 32768), kv=_log(rng, 1, 4096))
            if c["q"] <= c["kv"] and work(c)["flops"] <= 4 * 128 * 32 * 2048 * 16384 and work(c)["bytes"] <= 1 << 30:
                return c
        else:
            kind = rng.choice(["decode", "decode", "chunk"])
            c = dict(base, kind=kind, B=_log(rng, 1, 64 if kind == "decode" else 4),
                     q=1 if kind == "decode" else _log(rng, 2, 1024), kv=_log(rng, 64, 131072), k=_log(rng, FIRST + LAST, 64))
            rows = _rows(c)
            if c["q"] > c["kv"]:
                continue
            if op == "select_blocks":
                if (c["kv"] > 2 * c["k"] * c["page"] and sum(rows[1]) // c["page"] * Hkv * D <= 1 << 25
                        and sum(rows[0]) * c["kv"] // c["page"] * Hkv * D <= 1021 * 1024 * 2 * 128):
                    return c
            elif (c["B"] * c["kv"] * Hkv * D <= 1 << 30
                  and sum(rows[0]) * c["k"] * c["page"] * c["Hq"] * D <= 509 * 40 * 32 * 32 * 128):
                return c


def _rows(case):
    """New and cached tokens of every sequence (of paged_attention: cached ones behind the prefix)."""
    r = random.Random(case["lens"])
    B, q, kv = case["B"], case["q"], case["kv"]
    if case["kind"] == "decode":  # one token each; the first cache is full, the others anywhere
        return [1] * B, [kv] + [r.randint(1, kv) for _ in range(B - 1)]
    if case["op"] in ("paged_append", "select_blocks", "sparse_attention"):  # q tokens in all, cut anywhere
        cuts = [0] + sorted(r.randint(0, q) for _ in range(B - 1)) + [q]
        lq = [b - a for a, b in zip(cuts, cuts[1:])]
        if case["kind"] == "prompt":
            return lq, list(lq)
        return lq, [max(n, kv if b == 0 else r.randint(1, kv)) for b, n in enumerate(lq)]
    lq = [q] + [r.randint(1, q) for _ in range(B - 1)]
    return lq, [kv] + [r.randint(n, kv) for n in lq[1:]]


def _groups(case):
    """First sequence of every group and one past the last, and the groups' prefix lengths."""
    r = random.Random(case["lens"] + 1)
    B, n = case["B"], case["groups"]
    cu = [0] + sorted(r.sample(range(1, B), n - 1)) + [B]
    return cu, [case["prefix"]] + [r.randint(0, case["prefix"]) for _ in range(n - 1)]


FIRST, LAST = 1, 2  # pages at a context's beginning and end that every token selects


# ------------------------------------------------------------------ the least work
def work(case):
    lq, lk = _rows(case)
    T, Hq, Hkv, D, S = sum(lq), case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "paged_append":
        n = T * (Hq + 2 * Hkv) * D
        pages = sum((b - 1) // S - (b - a) // S + 1 for a, b in zip(lq, lk) if a)
        return dict(bytes=4 * n + 4 * T * case["R"] + 4 * T + 4 * pages * Hkv * D,
                    flops=6 * T * (Hq + Hkv) * D)
    if case["op"] == "paged_attention":
        cu, pre = _groups(case)
        seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
        seen += sum(p * sum(lq[i:j]) for p, i, j in zip(pre, cu, cu[1:]))
        return dict(bytes=2 * D * (2 * T * Hq + 2 * (sum(lk) + sum(pre)) * Hkv), flops=4 * D * Hq * seen)
    blocks = [-(-n // S) for n in lk]
    if case["op"] == "select_blocks":
        return dict(bytes=2 * D * (T * Hq + 2 * sum(blocks) * Hkv) + 4 * T * Hkv * case["k"],
                    flops=4 * D * Hkv * sum(a * n for a, n in zip(lq, blocks)))
    # a sequence reads at least the pages of one token, and its new tokens' own
    least = sum(min(b, max(min(case["k"], n) * S, a)) for a, b, n in zip(lq, lk, blocks))
    seen = sum(a * min(case["k"] * S, b) for a, b in zip(lq, lk))
    return dict(bytes=2 * D * (2 * T * Hq + 2 * least * Hkv) + 4 * T * Hkv * case["k"], flops=4 * D * Hq * seen)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, Hq, Hkv, D, S = (case[n] for n in ("op", "Hq", "Hkv", "D", "page"))
    lq, lk = _rows(case)
    B, T = case["B"], sum(lq)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) * std

    def ints(a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    # the page table: every sequence's pages anywhere in the pool; those of a shared prefix in several tables
    cu, pre = _groups(case) if op == "paged_attention" else (list(range(B + 1)), [0] * B)
    total = list(lk)
    for p, i, j in zip(pre, cu, cu[1:]):
        for b in range(i, j):
            total[b] += p
    need, shared = 0, []
    for p, i, j in zip(pre, cu, cu[1:]):
        shared.append(p // S)
        need += p // S + sum(-(-total[b] // S) - p // S for b in range(i, j))
    pages = torch.randperm(need + 1, generator=g, device="cuda").int()
    width = max(-(-n // S) for n in total)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    at = 0
    for s, i, j in zip(shared, cu, cu[1:]):
        table[i:j, :s] = pages[at:at + s]
        at += s
        for b in range(i, j):
            n = -(-total[b] // S) - s
            table[b, s:s + n] = pages[at:at + n]
            at += n
    ends = [0]
    for n in lq:
        ends.append(ends[-1] + n)
    st = dict(case=case, lq=lq, lk=total, q0=ends, table=table, cu=ints(ends), len=ints(total), n_pages=need + 1,
              most=(max(lq), max(lk)))
    if op == "paged_append":
        qkv = normal(T, Hq + 2 * Hkv, D, std=3.0)
        R = case["R"]
        P = max(total)
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * inv
        cache = normal(need + 1, S, 2 * Hkv, D)
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], kc=cache[:, :, :Hkv], vc=cache[:, :, Hkv:],
                  bounds=torch.stack([cache[:, :, :Hkv].amin(1), cache[:, :, :Hkv].amax(1)], 1).contiguous(),
                  qw=1 + 0.1 * torch.randn(D, generator=g, device="cuda") if case["norm"] else None,
                  kw=1 + 0.1 * torch.randn(D, generator=g, device="cuda") if case["norm"] else None,
                  cs=torch.cat([ang.cos(), ang.sin()], 1).float(),
                  q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"))
        return st
    st["q"] = normal(T, Hq, D, std=2.0)
    if op == "select_blocks":
        # pages that hold similar keys: a centre each, and the spread of a page's keys around it
        mid, spread = normal(need + 1, Hkv, D), normal(need + 1, Hkv, D, std=0.5).abs() + 1
        st["bounds"] = torch.stack([mid - spread, mid + spread], 1).contiguous()
    else:
        cache = normal(need + 1, S, 2 * Hkv, D)
        st.update(kc=cache[:, :, :Hkv], vc=cache[:, :, Hkv:],
                  out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"))
    if op == "paged_attention":
        st.update(group=ints(cu), prefix=ints(pre), max_prefix=max(pre))
    if op == "sparse_attention":
        st["blocks"] = _draw_blocks(case, lq, total, g)
    if own:
        from mxfp4_routed_expert_moe_amd import paged as P
        if op == "paged_attention":
            st["ws"] = P.paged_attention_workspace(st["q"], st["kc"], B, *st["most"], n_groups=case["groups"],
                                                   max_prefix=st["max_prefix"])
        elif op == "sparse_attention":
            st["ws"] = P.paged_attention_workspace(st["q"], st["kc"], B, *st["most"], n_blocks=case["k"])
        else:
            st["ws"] = P.select_blocks_workspace(st["q"], st["bounds"], B, *st["most"], S)
            st["blocks"] = torch.empty(T, Hkv, case["k"], dtype=torch.int32, device="cuda")
    return st


def _draw_blocks(case, lq, lk, g):
    """Selections as neighbouring tokens make them: the first page, the last two, and pages whose noisy rank among a
    sequence's is high, with most of the noise shared by 64 neighbours."""
    S, Hkv, k = case["page"], case["Hkv"], case["k"]
    out = []
    for n, m in zip(lq, lk):
        blocks = -(-m // S)
        last = (torch.arange(m - n, m, device="cuda") // S)[:, None, None]
        rank = torch.randn(-(-n // 64), Hkv, blocks, generator=g, device="cuda").repeat_interleave(64, 0)[:n]
        rank = rank + 0.1 * torch.randn(n, Hkv, blocks, generator=g, device="cuda")
        i = torch.arange(blocks, device="cuda")
        rank = torch.where((i < FIRST) | (i > last - LAST), torch.full_like(rank, 100.0), rank)
        rank = torch.where(i > last, torch.full_like(rank, -100.0), rank)
        pick = rank.topk(min(k, blocks), -1).indices
        pick = torch.where(pick > last, torch.full_like(pick, blocks), pick).sort(-1).values
        pick = torch.where(pick == blocks, torch.full_like(pick, -1), pick).int()
        out.append(torch.nn.functional.pad(pick, (0, k - pick.shape[-1]), value=-1))
    return torch.cat(out).contiguous()


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"paged_append": _plain_append, "paged_attention": _plain_attention, "select_blocks": _plain_select,
                "sparse_attention": _plain_sparse}[op](st)
    from mxfp4_routed_expert_moe_amd import paged as P
    at = (st["cu"], st["len"], st["table"])
    if op == "paged_append":
        P.paged_append(st["k"], st["v"], st["kc"], st["vc"], *at, q=st["q"], q_out=st["q_out"], bounds=st["bounds"],
                       q_weight=st["qw"], k_weight=st["kw"], norm=case["norm"], cos_sin=st["cs"],
                       rot_offset=_tail(case), interleaved=case["interleaved"])
        return st["q_out"], st["kc"], st["vc"], st["bounds"]
    if op == "paged_attention":
        return P.paged_attention(st["q"], st["kc"], st["vc"], *at, *st["most"], cu_group=st["group"],
                                 prefix_len=st["prefix"], max_prefix=st["max_prefix"], out=st["out"], ws=st["ws"])
    if op == "select_blocks":
        return P.select_blocks(st["q"], st["bounds"], *at, *st["most"], case["page"], case["k"], first=FIRST, last=LAST,
                               blocks=st["blocks"], ws=st["ws"])
    return P.paged_attention(st["q"], st["kc"], st["vc"], *at, *st["most"], blocks=st["blocks"], out=st["out"],
                             ws=st["ws"])


def _tail(case):
    """Where the rotated part of a head begins."""
    return case["D"] - case["R"] if case["tail"] else 0


def _tokens(st):
    """Sequence and position of every new token."""
    lq = torch.tensor(st["lq"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(st["lq"]), device="cuda"), lq)
    first = torch.tensor([m - n - a for n, m, a in zip(st["lq"], st["lk"], st["q0"])], device="cuda")
    return seq, torch.arange(len(seq), device="cuda") + first[seq]


def _plain_append(st):
    case = st["case"]
    S, R, off = case["page"], case["R"], _tail(case)
    seq, pos = _tokens(st)
    page, slot = st["table"][seq, pos // S].long(), pos % S
    c, s = st["cs"][pos][:, None, :R // 2], st["cs"][pos][:, None, R // 2:]

    def turn(x, w):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        r = x[..., off:off + R]
        a, b = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., :R // 2], r[..., R // 2:])
        ra, rb = a * c - b * s, b * c + a * s
        r = torch.stack([ra, rb], -1).flatten(-2) if case["interleaved"] else torch.cat([ra, rb], -1)
        return torch.cat([x[..., :off], r, x[..., off + R:]], -1).bfloat16()

    st["q_out"].copy_(turn(st["q"], st["qw"]))
    k = turn(st["k"], st["kw"])
    st["kc"][page, slot] = k
    st["vc"][page, slot] = st["v"]
    low, high = st["bounds"][:, 0].float(), st["bounds"][:, 1].float()
    fresh = page[slot == 0]  # pages that begin anew
    low[fresh], high[fresh] = float("inf"), float("-inf")
    at = page[:, None, None].expand(k.shape)
    low.scatter_reduce_(0, at, k.float(), "amin")
    high.scatter_reduce_(0, at, k.float(), "amax")
    st["bounds"].copy_(torch.stack([low, high], 1))
    return st["q_out"], st["kc"], st["vc"], st["bounds"]


def _plain_attention(st):
    case = st["case"]
    Hq, Hkv, D, S = (case[n] for n in ("Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = st["out"]
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        pages = st["table"][b, :-(-m // S)].long()
        k = st["kc"][pages].flatten(0, 1)[:m].float().permute(1, 2, 0).contiguous()  # [Hkv, D, m]
        v = st["vc"][pages].flatten(0, 1)[:m].float().transpose(0, 1).contiguous()   # [Hkv, m, D]
        q = st["q"][a:a + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        z = torch.matmul(q, k).view(Hkv, G, n, m) * (1 / math.sqrt(D))
        if n > 1:
            seen = torch.arange(m, device="cuda") <= torch.arange(n, device="cuda")[:, None] + (m - n)
            z = z.masked_fill(~seen, float("-inf"))
        p = torch.exp(z - z.amax(-1, keepdim=True))
        o = torch.matmul(p.view(Hkv, G * n, m), v).view(Hkv, G, n, D) / p.sum(-1, keepdim=True)
        out[a:a + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).bfloat16()
    return out


def _plain_select(st):
    case = st["case"]
    Hkv, D, S, k = (case[n] for n in ("Hkv", "D", "page", "k"))
    res = []
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        if n == 0:
            continue
        blocks = -(-m // S)
        bounds = st["bounds"][st["table"][b, :blocks].long()].double()   # [blocks, 2, Hkv, D]
        q = st["q"][a:a + n].double().view(n, Hkv, -1, D)
        up, down = q.clamp_min(0).sum(2).transpose(0, 1), q.clamp_max(0).sum(2).transpose(0, 1)
        score = (torch.matmul(up, bounds[:, 1].permute(1, 2, 0).contiguous())
                 + torch.matmul(down, bounds[:, 0].permute(1, 2, 0).contiguous())).transpose(0, 1)  # [n, Hkv, blocks]
        score = torch.where(torch.isfinite(score), score, torch.full_like(score, 1e300))
        last = (torch.arange(m - n, m, device="cuda") // S)[:, None, None]
        i = torch.arange(blocks, device="cuda")
        score = torch.where((i < FIRST) | (i > last - LAST), torch.full_like(score, float("inf")), score)
        score = torch.where(i > last, torch.full_like(score, float("-inf")), score)
        pick = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
        pick = torch.where(pick > last, torch.full_like(pick, blocks), pick).sort(-1).values
        pick = torch.where(pick == blocks, torch.full_like(pick, -1), pick).int()
        res.append(torch.nn.functional.pad(pick, (0, k - pick.shape[-1]), value=-1))
    return torch.cat(res)


def _plain_sparse(st):
    case = st["case"]
    Hq, Hkv, D, S, k = (case[n] for n in ("Hq", "Hkv", "D", "page", "k"))
    G = Hq // Hkv
    seq, pos = _tokens(st)
    head = torch.arange(Hkv, device="cuda")[:, None]
    step = max(1, (1 << 27) // (Hkv * k * S * D))  # half a GiB of gathered keys at a time
    for t in range(0, len(seq), step):
        ids = st["blocks"][t:t + step].long()                                     # [n, Hkv, k]
        n = ids.shape[0]
        page = st["table"][seq[t:t + step, None, None], ids.clamp_min(0)].long()
        kk = st["kc"].transpose(1, 2)[page, head].float().view(n, Hkv, k * S, D)
        vv = st["vc"].transpose(1, 2)[page, head].float().view(n, Hkv, k * S, D)
        key = (ids[..., None] * S + torch.arange(S, device="cuda")).view(n, Hkv, 1, k * S)
        seen = (key >= 0) & (key <= pos[t:t + step, None, None, None])
        q = st["q"][t:t + step].float().view(n, Hkv, G, D)
        z = torch.matmul(q, kk.transpose(2, 3).contiguous()) * (1 / math.sqrt(D))
        z = z.masked_fill(~seen, float("-inf"))
        p = torch.exp(z - z.amax(-1, keepdim=True))
        o = torch.matmul(p, vv) / p.sum(-1, keepdim=True)
        st["out"][t:t + step] = o.view(n, Hq, D).bfloat16()
    return st["out"]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"paged_append": _exact_append, "paged_attention": _exact_attention, "select_blocks": _exact_select,
            "sparse_attention": _exact_sparse}[case["op"]](st)


def _exact_append(st):
    case = st["case"]
    S, R = case["page"], case["R"]
    half = torch.arange(R // 2, device="cuda")
    i, j = (2 * half, 2 * half + 1) if case["interleaved"] else (half, half + R // 2)
    i, j = i + _tail(case), j + _tail(case)
    kc, vc, bounds = st["kc"].double(), st["vc"].double(), st["bounds"].double()
    q_out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        turn = torch.complex(st["cs"][m - n:m, None, :R // 2].double(), st["cs"][m - n:m, None, R // 2:].double())
        new = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            y = x[a:a + n].double()
            if case["norm"]:
                y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6) * w.double()
            z = torch.complex(y[..., i], y[..., j]) * turn
            y = y.clone()
            y[..., i], y[..., j] = z.real, z.imag
            new.append(y)
        q_out[a:a + n] = new[0]
        p = m - n
        while p < m:  # page by page
            page, end = int(st["table"][b, p // S]), min(m, (p // S + 1) * S)
            rows = new[1][p - m + n:end - m + n]
            kc[page, p % S:p % S + end - p] = rows
            vc[page, p % S:p % S + end - p] = st["v"][a + p - m + n:a + end - m + n].double()
            if p % S:
                rows = torch.cat([rows, bounds[page]])
            bounds[page, 0], bounds[page, 1] = rows.min(0).values, rows.max(0).values
            p = end
    return q_out, kc, vc, bounds


def _exact_attention(st):
    case = st["case"]
    G, S = case["Hq"] // case["Hkv"], case["page"]
    if sum(n * m for n, m in zip(st["lq"], st["lk"])) * case["Hq"] * case["D"] > 4e11:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        key = torch.arange(m, device="cuda")
        page, slot = st["table"][b, key // S].long(), key % S
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(case["Hkv"]):
            k, v = st["kc"][page, slot, h].double(), st["vc"][page, slot, h].double()
            for r in range(h * G, h * G + G):
                z = (k @ st["q"][a:a + n, r].double().t()).t() / math.sqrt(case["D"])
                out[a:a + n, r] = torch.softmax(z.masked_fill(hidden, float("-inf")), -1) @ v
    return out


def _exact_select(st):
    case = st["case"]
    S, k, G = case["page"], case["k"], case["Hq"] // case["Hkv"]
    ids = torch.full((sum(st["lq"]), case["Hkv"], k), -1, dtype=torch.int32, device="cuda")
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        blocks = -(-m // S)
        bounds = st["bounds"][st["table"][b, :blocks].long()].double()
        step = max(1, (1 << 26) // (blocks * case["D"]))
        for h in range(case["Hkv"]):
            low, high = bounds[:, 0, h], bounds[:, 1, h]
            for t in range(0, n, step):
                e = min(n, t + step)
                score = torch.zeros(e - t, blocks, dtype=torch.float64, device="cuda")
                for r in range(h * G, h * G + G):
                    q = st["q"][a + t:a + e, r].double()[:, None]
                    score += torch.maximum(q * low, q * high).sum(-1)
                score[~torch.isfinite(score)] = 1e300
                last = torch.arange(m - n + t, m - n + e, device="cuda") // S
                score[:, :FIRST] = float("inf")
                for back in range(LAST):
                    rows = torch.arange(e - t, device="cuda")[last >= back]
                    score[rows, last[last >= back] - back] = float("inf")
                score[torch.arange(blocks, device="cuda") > last[:, None]] = float("-inf")
                order = torch.argsort(-score, dim=-1, stable=True)[:, :k]
                marks = torch.zeros(e - t, blocks, dtype=torch.bool, device="cuda").scatter_(1, order, True)
                marks &= torch.arange(blocks, device="cuda") <= last[:, None]
                place = marks.cumsum(1) - 1
                row, col = marks.nonzero(as_tuple=True)
                ids[a + t + row, h, place[row, col]] = col.int()
    return ids


def _exact_sparse(st):
    case = st["case"]
    G, S = case["Hq"] // case["Hkv"], case["page"]
    if sum(n * m for n, m in zip(st["lq"], st["lk"])) * case["Hq"] * case["D"] > 4e11:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, (a, n, m) in enumerate(zip(st["q0"], st["lq"], st["lk"])):
        key = torch.arange(m, device="cuda")
        page, slot = st["table"][b, key // S].long(), key % S
        for h in range(case["Hkv"]):
            ids = st["blocks"][a:a + n, h].long()
            seen = torch.zeros(n, -(-m // S) + 1, dtype=torch.bool, device="cuda").scatter_(1, ids + 1, True)
            seen = seen[:, 1:][:, key // S] & (key <= torch.arange(m - n, m, device="cuda")[:, None])
            k, v = st["kc"][page, slot, h].double(), st["vc"][page, slot, h].double()
            for r in range(h * G, h * G + G):
                z = (k @ st["q"][a:a + n, r].double().t()).t() / math.sqrt(case["D"])
                out[a:a + n, r] = torch.softmax(z.masked_fill(~seen, float("-inf")), -1) @ v
    return out
