"""PagedAttentionBlock on the GPU: prompts, forks, chunks and single tokens over its pages, against the references over
what the pages then hold and against the block over a contiguous cache; selected pages; and the example, eager steps
against graph replays."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from mxfp4_routed_expert_moe_amd import block as K  # noqa: E402
from tests import paged_reference as PR  # noqa: E402
from tests.test_paged_gpu import BF, U, _check, _np  # noqa: E402

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[paged block]", *a, flush=True)


def _blocks(Hq=8, Hkv=2, D=64, hidden=272, max_seqs=4, max_len=400, max_tokens=500, seed=3, **kw):
    """The paged block, and one over rows with the same weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [torch.randn(n, k, generator=g, device="cuda") * k ** -0.5 for n, k in (((Hq + 2 * Hkv) * D, hidden), (hidden, Hq * D))]
    qw, kw_ = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")
    args = (*K.quantise_weight(w[0]), *K.quantise_weight(w[1]), Hq, Hkv, D, K.rope_table(max_len, D), qw, kw_)
    size = dict(max_seqs=max_seqs, max_len=max_len, max_tokens=max_tokens)
    return K.PagedAttentionBlock(*args, **size, n_pages=kw.pop("n_pages", 100), **kw), K.AttentionBlock(*args, **size)


def _x(T, hidden, seed):
    return torch.randn(T, hidden, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def _verify(b, new, plan):
    """The last call's attention against the reference over the pages."""
    T, cu = sum(new), np.r_[0, np.cumsum(new)]
    lens = plan.kv_len.tolist()
    seqs = [(int(cu[s]), n, lens[s] if n else 0) for s, n in enumerate(new)]
    table = b.table.cpu().numpy()
    blocks = b.blocks[:T].cpu().numpy() if b._selects(plan) else None
    if blocks is not None:
        n, first, last = b.select
        assert np.array_equal(blocks, PR.select(_np(b.qkv[:T, :b.Hq]), _np(b.bounds), table, seqs, b.page_size, n, first, last))
    see = PR.visible(seqs, table, b.page_size, b.n_pages, b.Hkv, blocks)
    _check(b.o[:T], None, _np(b.qkv[:T, :b.Hq]), _np(b.k_pages), _np(b.v_pages), table, seqs, see, b.D ** -0.5)
    for s, (q0, n, m) in enumerate(seqs):  # the keys and values of the call are in their slots
        for i in range(n):
            page, slot = table[s, (m - n + i) // b.page_size], (m - n + i) % b.page_size
            assert torch.equal(b.v_pages[page, slot], b.qkv[q0 + i, b.Hq + b.Hkv:])


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (4, 4, 128, 64), (4, 1, 256, 32)])
def test_prompts_forks_chunks_and_steps(Hq, Hkv, D, page):
    b, rows = _blocks(Hq, Hkv, D, seed=D, page_size=page)
    step = None
    # new tokens per sequence; ("fork", src, dst); None: the last plan advanced
    calls = [[150, 0, 0, 17], ("fork", 0, 1), ("fork", 0, 2), [1, 1, 1, 1], [3, 0, 40, 1], [0, 20, 1, 0], ("steps", [1, 1, 1, 1]), None, None]
    for i, new in enumerate(calls):
        _say("call", Hq, Hkv, D, page, new)
        if isinstance(new, tuple) and new[0] == "fork":
            b.fork(*new[1:])
            src, dst = (slice(rows.max_len * s, rows.max_len * (s + 1)) for s in new[1:])
            rows.cache[dst] = rows.cache[src]
            rows.lens[new[2]] = rows.lens[new[1]]
            continue
        if new is None:
            step.advance()
            other.advance()  # noqa: F821
            new = [1, 1, 1, 1]
        else:
            bound = 300 if isinstance(new, tuple) else None
            new = new[1] if isinstance(new, tuple) else new
            step, other = b.plan(new, max_kv=bound), rows.plan(new, max_kv=bound)
        x = _x(sum(new), 272, 10 + i)
        y = b.forward(x, step, b.workspace(step)).clone()
        assert step.kv_len.tolist() == other.kv_len.tolist()
        _verify(b, new, step)
        # The same queries and keys, bit by bit; each attention is within its bound of the exact one (see the tests of the
        # operators), so what is left is that both were given the same work: outputs of a block differ by a small part of themselves.
        z = rows.forward(x, other)
        assert torch.equal(b.qkv[:sum(new), :Hq], rows.qkv[:sum(new), :Hq])
        assert torch.equal(b.v_pages[b.table[0, 0].item(), 0], rows.cache[0, Hkv:])
        d = torch.linalg.vector_norm(y.float() - z.float()) / torch.linalg.vector_norm(z.float())
        # per element of o: each side off by at most 3.1 u sum p |v| (u |o| + 2 u A, sums far below); E4M3 of o rounds by 2^-4 at most
        # where the two sides fall on different codes
        assert d <= 2 * (3.1 * U + 2.0 ** -4)
    assert step.group is not None


def test_selected_pages():
    b, _ = _blocks(8, 2, 64, page_size=16, select=(5, 1, 2))
    _say("selected pages")
    b.forward(_x(290, 272, 1), p := b.plan([200, 90]))
    _verify(b, [200, 90], p)
    b.fork(0, 2)
    step = b.plan([1, 1, 1], max_kv=240)
    ws = b.workspace(step)
    for i in range(12):
        b.forward(_x(3, 272, 20 + i), step, ws)
        _verify(b, [1, 1, 1], step)
        step.advance()


@pytest.mark.parametrize("select", [None, (6, 1, 2)])
def test_example(select):
    """Every replay gives the eager step's bits."""
    _say("example", select)
    eager, replayed = K.paged_example(hidden=256, q_heads=4, kv_heads=2, head_dim=64, prompt=200, samples=3, steps=5, select=select)
    assert len(eager) == 5 and all(torch.isfinite(a).all() for a in eager)
    for a, r in zip(eager, replayed):
        assert torch.equal(a, r)


def test_replays_past_the_pages_store_nothing():
    """A graph replayed more often than its plan has pages for leaves every other sequence's pages alone."""
    _say("past the pages")
    b, _ = _blocks(4, 2, 64, page_size=16, n_pages=9, max_len=400)
    b.forward(_x(60, 272, 1), b.plan([30, 30]))
    step = b.plan([1, 0], max_kv=31)
    x = _x(1, 272, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b._enqueue(x, step, None)
    torch.cuda.current_stream().wait_stream(side)
    ws = b.workspace(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b._enqueue(x, step, ws)
        step._shift()
    torch.cuda.synchronize()
    own = b.pages[0]
    before = b.cache.clone()
    for _ in range(40):
        graph.replay()
    torch.cuda.synchronize()
    others = [p for p in range(9) if p not in own]
    assert torch.equal(b.cache[others], before[others])


def test_replays_of_a_forked_prompt_leave_its_pages_alone():
    """A captured prompt that is replayed after a fork stores nothing to the pages that both sequences hold; its own last page, and
    after the other sequence has gone all of them, it writes."""
    _say("replays after a fork")
    b, _ = _blocks(4, 2, 64, page_size=16, max_seqs=2, n_pages=20, max_len=200)
    x, prompt = _x(60, 272, 1), b.plan([60])
    ws = b.workspace(prompt)
    b.forward(x, prompt, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(x, prompt, ws)
    b.fork(0, 1)
    with pytest.raises(ValueError):
        b.forward(x, prompt, ws)
    shared, last = b.pages[0][:3], b.pages[0][3]
    before = b.cache.clone()
    x.copy_(_x(60, 272, 2))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        others = [p for p in range(20) if p != last]
        assert torch.equal(b.cache[others], before[others])
    assert not torch.equal(b.cache[last], before[last])
    step = b.plan([0, 1])
    b.forward(_x(1, 272, 3), step)
    _verify(b, [0, 1], step)
    b.reset(1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(b.cache[shared], before[shared])
    _verify(b, [60], prompt)
