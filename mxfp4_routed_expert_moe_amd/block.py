"""The attention half of a decoder block over a key/value cache, in front of the
MoE layer: the operators of `attention` in the order in which a model runs them.

    qkv = x W_qkv^T                  fp8_linear
    q, k normed and rotated in qkv   qk_norm_rope, in place
    k | v to the cache               one row copy
    o = softmax(q K^T) V             attention over the cache
    y = o W_out^T                    fp8_linear

`AttentionBlock.plan` says which tokens a call brings: whole prompts, chunks of
prompts, single tokens, or a mixture.  `AttentionBlock.forward` then only
enqueues kernels on the current stream, so a single-token step and
`Plan.advance` can be captured into a HIP graph and replayed once per token.

`python -m mxfp4_routed_expert_moe_amd.block` runs a small decoder block: three
prompts, then single-token steps, eager and as a graph.
"""
from __future__ import annotations

import torch

from . import attention as A


class Plan:
    """The tokens of one call, sequence after sequence, and where they go.

    cu_q, kv_len, positions and rows are int32 (rows: int64) device tensors,
    counts holds positions and kv_len, last the last cache row of each token's
    sequence; max_q and max_kv bound the sequences' new tokens and cached
    lengths.  The block that made the plan knows how many tokens each sequence
    holds; forward, advance and replayed keep that in step."""

    def __init__(self, block, number, new, cu_q, counts, rows, last, max_q, max_kv, longest):
        self.block, self.number, self.new = block, number, list(new)
        self.cu_q, self.counts, self.rows, self.last = cu_q, counts, rows, last
        self.positions, self.kv_len = counts[:rows.numel()], counts[rows.numel():]
        self.max_q, self.max_kv = max_q, max_kv
        self.steps = 0  # how often it was advanced
        self.cancelled = False
        self.longest = longest  # of its sequences, with the plan's tokens

    def advance(self):
        """The same call one token later (plans of at most one token per
        sequence): three small kernels on the current stream.  The step before counts
        as run; the one that is announced counts for later plans once it has
        run, by forward, or by the next advance after a graph's replay.  The last
        step is the one whose longest sequence holds max_kv tokens."""
        self.replayed(1)
        self._shift()

    def _shift(self):
        """The device's part of advance.  Replays that pass the cache's end, which no
        check on the host sees, write the last row of their own sequence."""
        self.counts.add_(1)
        self.rows.add_(1)
        torch.minimum(self.rows, self.last, out=self.rows)

    def replayed(self, steps: int):
        """Note `steps` replays of a HIP graph that holds forward and then advance();
        called before them, it refuses those that would pass max_kv."""
        if any(n > 1 for n in self.new):
            raise ValueError("a plan of more than one token per sequence cannot be advanced")
        if steps < 0:
            raise ValueError(f"steps must not be negative, got {steps}")
        self._check(advance=True)
        if steps == 0:
            return
        if self.longest + steps - 1 > self.max_kv:
            raise ValueError(f"the plan's sequences would hold {self.longest + steps - 1} tokens, its bound is {self.max_kv}")
        for b in self._sequences():
            self.block.lens[b] += steps
            self.block._announced[b] = self.block.lens[b]
        self._ran()
        self.steps += steps
        self.longest += steps

    def cancel(self):
        """Give the plan's tokens back: it will not run.  Only before it has run, and before
        the plans that were made after it for its sequences are cancelled or reset."""
        at = [b for b in self._sequences() if self.number > self.block._since[b]]
        if self.cancelled or any(self.block._unrun[b][-1:] != [self.number] for b in at):
            raise ValueError("the plan has run, was cancelled, or is not the last one of its sequences")
        self.cancelled = True
        for b in at:
            self.block.lens[b] -= self.new[b]
            self.block._unrun[b].pop()
            self.block._owner[b] = 0

    def _sequences(self):
        """The sequences that the plan brings tokens to."""
        return [b for b, n in enumerate(self.new) if n]

    def _check(self, advance=False):
        """Whether the plan's step can run now: the plans before it have, and, once it is
        advanced, no later plan has brought the token that would be its next."""
        for b in self._sequences():
            if self.cancelled or self.number <= self.block._since[b]:
                raise ValueError(f"the plan was cancelled, or sequence {b} reset: make a new plan")
            if self.block._unrun[b] and self.block._unrun[b][0] < self.number:
                raise ValueError(f"a plan made before this one for sequence {b} has not run: run it, or cancel it")
            if (self.steps or advance) and self.block._owner[b] != self.number:
                raise ValueError(f"a later plan has brought tokens to sequence {b}: make a new plan")

    def _ran(self):
        for b in self._sequences():
            if self.number in self.block._unrun[b]:
                self.block._unrun[b].remove(self.number)


class AttentionBlock:
    """Weights, cache and buffers of one block's attention.

    w_qkv [(q_heads + 2 kv_heads) D, hidden] and w_out [hidden, q_heads D]: E4M3
    with the scales of fp8_linear.  cos_sin [n_positions, rot_dim]; q_weight,
    k_weight: float32 [D] or None.  The cache holds max_seqs sequences of up to
    max_len tokens; a row of it is the token's key heads, then its value heads.
    max_tokens: the most tokens of one call."""

    def __init__(self, w_qkv, qkv_scale, w_out, out_scale, q_heads: int, kv_heads: int, head_dim: int, cos_sin,
                 q_weight=None, k_weight=None, *, max_seqs: int, max_len: int, max_tokens: int, rot_offset=0,
                 interleaved=False, eps=1e-6):
        self.w_qkv, self.qkv_scale, self.w_out, self.out_scale = w_qkv, qkv_scale, w_out, out_scale
        self.Hq, self.Hkv, self.D = q_heads, kv_heads, head_dim
        self.hidden = w_qkv.shape[1]
        if w_qkv.shape[0] != (q_heads + 2 * kv_heads) * head_dim:
            raise ValueError(f"w_qkv must have {(q_heads + 2 * kv_heads) * head_dim} rows, got {w_qkv.shape[0]}")
        if tuple(w_out.shape) != (self.hidden, q_heads * head_dim):
            raise ValueError(f"w_out must have shape {(self.hidden, q_heads * head_dim)}, got {tuple(w_out.shape)}")
        if max_len > cos_sin.shape[0]:
            raise ValueError(f"max_len {max_len} exceeds the {cos_sin.shape[0]} positions of cos_sin")
        self.cos_sin, self.q_weight, self.k_weight = cos_sin, q_weight, k_weight
        self.rope = dict(rot_offset=rot_offset, interleaved=interleaved, eps=eps)
        self.max_seqs, self.max_len, self.max_tokens = max_seqs, max_len, max_tokens
        dev, bf16 = w_qkv.device, torch.bfloat16
        self.lens = [0] * max_seqs  # tokens that each sequence holds once its plans and their announced steps have run
        self._announced = [None] * max_seqs  # what lens is with a step that was announced and has not run
        self._owner = [0] * max_seqs  # the number of the last plan that brought tokens
        self._unrun = [[] for _ in range(max_seqs)]  # the numbers of the plans that have not run
        self._since = [0] * max_seqs  # plans up to this number ended with a reset
        self._plans = 0
        self.cache = torch.empty((max_seqs * max_len, 2 * kv_heads, head_dim), dtype=bf16, device=dev)
        self.kv_start = torch.arange(0, max_seqs * max_len, max_len, dtype=torch.int32, device=dev)
        self.qkv = torch.empty((max_tokens, q_heads + 2 * kv_heads, head_dim), dtype=bf16, device=dev)
        self.o = torch.empty((max_tokens, q_heads, head_dim), dtype=bf16, device=dev)
        self.y = torch.empty((max_tokens, self.hidden), dtype=bf16, device=dev)
        self.ws = A.fp8_linear_workspace(max_tokens, max(w_qkv.shape[0], self.hidden),
                                         max(self.hidden, w_out.shape[1]), dev)

    def held(self, b: int) -> int:
        """Tokens of sequence b that count for the next plan: those of all plans made so
        far, and of the steps of advanced plans that have run."""
        return self.lens[b] - (self._announced[b] == self.lens[b])

    def reset(self, b=None):
        """Forget the tokens of sequence b (None: of all) and the plans that bring it some: its next
        plan begins at position 0."""
        if b is not None and not 0 <= b < self.max_seqs:
            raise ValueError(f"there are {self.max_seqs} sequences, got {b}")
        self._plans += 1
        for s in range(self.max_seqs) if b is None else (b,):
            self.lens[s], self._announced[s], self._owner[s] = 0, None, 0
            self._unrun[s], self._since[s] = [], self._plans

    def plan(self, new, max_kv=None) -> Plan:
        """A call that brings new[b] tokens to sequence b, after those it holds (host
        list; fewer entries than max_seqs: the first ones).  Plans run in the order in
        which they were made; one that is not to run is cancelled.  max_kv: the bound on the cached lengths of the sequences
        that get tokens, this call's by default; a plan that is to be advanced passes the one of its last step."""
        if len(new) > self.max_seqs or any(n < 0 for n in new):
            raise ValueError(f"new must hold up to {self.max_seqs} counts")
        if sum(new) > self.max_tokens:
            raise ValueError(f"{sum(new)} tokens, the block was built for {self.max_tokens}")
        held = [self.held(b) for b in range(len(new))]
        ends = [have + n for have, n in zip(held, new)]
        if any(e > self.max_len for e in ends):
            raise ValueError(f"a sequence would hold {max(ends)} tokens, the cache has room for {self.max_len}")
        longest = max((e for e, n in zip(ends, new) if n), default=0)
        if max_kv is None:
            max_kv = longest
        if not longest <= max_kv <= self.max_len:
            raise ValueError(f"max_kv must be {longest} to {self.max_len}, got {max_kv}")
        cu, pos, rows, last = [0], [], [], []
        for b, n in enumerate(new):
            cu.append(cu[-1] + n)
            pos.extend(range(held[b], ends[b]))
            rows.extend(range(b * self.max_len + held[b], b * self.max_len + ends[b]))
            last.extend([(b + 1) * self.max_len - 1] * n)
        dev = self.cache.device
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        i64 = lambda v: torch.tensor(v, dtype=torch.int64, device=dev)  # noqa: E731
        plan = Plan(self, self._plans + 1, new, i32(cu), i32(pos + ends), i64(rows), i64(last), max(new, default=0), max_kv,
                    longest)
        self._plans += 1
        for b, n in enumerate(new):
            if n:  # an announced step of a sequence without new tokens keeps its place
                self.lens[b], self._announced[b], self._owner[b] = ends[b], None, self._plans
                self._unrun[b].append(self._plans)
        return plan

    def workspace(self, plan: Plan):
        """The attention workspace of a plan, for callers that keep it."""
        n = plan.rows.numel()
        return A.attention_workspace(self.qkv[:n, :self.Hq], self.cache[:, :self.Hkv], plan.cu_q.numel() - 1,
                                     plan.max_q, plan.max_kv)

    def forward(self, x, plan: Plan, ws=None):
        """x bf16 [tokens of the plan, hidden] -> y of the same shape, a view of
        the block's buffer (valid until its next call)."""
        T = plan.rows.numel()
        if tuple(x.shape) != (T, self.hidden):
            raise ValueError(f"x must have shape {(T, self.hidden)}, got {tuple(x.shape)}")
        if T == 0:
            return self.y[:0]
        if plan.longest > plan.max_kv:
            raise ValueError(f"the plan was advanced to {plan.longest} tokens, its bound is {plan.max_kv}")
        plan._check()
        y = self._enqueue(x, plan, ws)
        plan._ran()
        for b in plan._sequences():
            if self._owner[b] == plan.number:
                self._announced[b] = None
        return y

    def _enqueue(self, x, plan: Plan, ws):
        """The device's part of forward."""
        T, Hq, Hkv = plan.rows.numel(), self.Hq, self.Hkv
        qkv, o, y = self.qkv[:T], self.o[:T], self.y[:T]
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        A.fp8_linear(x, self.w_qkv, self.qkv_scale, y=qkv.view(T, -1), ws=self.ws)
        A.qk_norm_rope(q, k, self.q_weight, self.k_weight, plan.positions, self.cos_sin, q_out=q, k_out=k, **self.rope)
        self.cache.index_copy_(0, plan.rows, qkv[:, Hq:])
        A.attention(q, self.cache[:, :Hkv], self.cache[:, Hkv:], plan.cu_q, plan.max_q,
                    kv_start=self.kv_start[:plan.cu_q.numel() - 1], kv_len=plan.kv_len, max_kv=plan.max_kv, out=o,
                    ws=ws)
        return A.fp8_linear(o.view(T, -1), self.w_out, self.out_scale, y=y, ws=self.ws)


# ---------------------------------------------------------------- example
def rope_table(n_positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos_sin of rotary positions: pair j turns by position * base^(-2 j / rot_dim)."""
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def quantise_weight(w):
    """float [N, K] -> (E4M3 codes [N, K], E8M0 scales [ceil(N / 128), ceil(K / 128)]):
    per 128 x 128 block the least power of two that brings its largest value
    to at most 448."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    padded = torch.zeros((nb * 128, kb * 128), dtype=torch.float32, device=w.device)
    padded[:N, :K] = w
    blocks = padded.view(nb, 128, kb, 128)
    top = blocks.abs().amax((1, 3)).clamp_min(2.0 ** -100)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    scale = torch.where(top > 448 * scale, 2 * scale, scale)
    codes = (blocks / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(nb * 128, kb * 128)[:N, :K].contiguous(), (torch.log2(scale) + 127).to(torch.uint8)


def example(hidden=1024, q_heads=8, kv_heads=2, head_dim=128, n_experts=16, inter=512, prompts=(70, 33, 5), steps=6,
            seed=7):
    """A decoder block (attention, then the MoE layer, each added to its input) on
    random weights: prompts, then single tokens fed back, eager and as a graph.
    -> (outputs of the eager steps, outputs of the graph's replays)."""
    from . import binding as B
    from . import workloads as WL

    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    w_qkv = quantise_weight(rand((q_heads + 2 * kv_heads) * head_dim, hidden) * hidden ** -0.5)
    w_out = quantise_weight(rand(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5)
    weights = 1 + 0.1 * rand(2, head_dim)
    cos_sin = rope_table(256, head_dim)
    experts = B.Experts.from_canonical(WL.make_experts(seed, n_experts + 1, hidden, inter), n_experts, hidden, inter)
    router = torch.from_numpy(WL.make_router(seed, hidden, n_experts)).cuda()
    x0 = rand(sum(prompts), hidden).bfloat16()

    def build():
        attn = AttentionBlock(*w_qkv, *w_out, q_heads, kv_heads, head_dim, cos_sin, weights[0], weights[1],
                              max_seqs=len(prompts), max_len=256, max_tokens=sum(prompts))
        moe = {T: B.MoeLayer(experts, T, 6, WL.ROUTE_SCALE, WL.CLAMP_LIMIT, router)
               for T in (sum(prompts), len(prompts))}

        def block(x, plan, ws):
            h = x + attn.forward(x, plan, ws)
            return h + moe[len(h)].forward(h.view(torch.int16)).view(torch.bfloat16)
        first = attn.plan(prompts)
        y = block(x0, first, attn.workspace(first))
        x = y[first.cu_q[1:].long() - 1].contiguous()  # each sequence's last token
        step = attn.plan([1] * len(prompts), max_kv=max(prompts) + steps)
        return block, x, step, attn.workspace(step)

    block, x, step, ws = build()
    eager = []
    for _ in range(steps):
        x = block(x, step, ws)
        step.advance()
        eager.append(x)

    block, x, step, ws = build()
    replayed = []
    start = [t.clone() for t in (x, step.positions, step.kv_len, step.rows)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # one step outside the graph: the library loads its kernels
        block(x, step, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(block(x, step, ws))
        step.advance()  # counts the first replay
    for t, v in zip((x, step.positions, step.kv_len, step.rows), start):
        t.copy_(v)
    step.replayed(steps - 1)
    for _ in range(steps):
        graph.replay()
        replayed.append(x.clone())
    torch.cuda.synchronize()
    return eager, replayed


if __name__ == "__main__":
    eager, replayed = example()
    for i, (a, b) in enumerate(zip(eager, replayed)):
        print(f"step {i}: {tuple(a.shape)} {a.dtype}, |y| {a.float().norm():.3f}; graph replay "
              + ("bit-identical" if torch.equal(a, b) else f"off by {(a.float() - b.float()).abs().max():.3g}"))
