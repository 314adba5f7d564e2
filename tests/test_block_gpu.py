"""AttentionBlock on the GPU: prompts, chunks and single tokens over its cache
against the operators called by hand and against the float64 references, its
refusals, and the example (eager steps against graph replays)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from mxfp4_routed_expert_moe_amd import attention as A  # noqa: E402
from mxfp4_routed_expert_moe_amd import block as K  # noqa: E402
from tests import attention_reference as R  # noqa: E402
from tests.test_attention_gpu import BF, U, _check_attention, _check_linear, _gpu, _np  # noqa: E402

pytestmark = pytest.mark.gpu


def _block(Hq=8, Hkv=2, D=64, hidden=272, max_seqs=4, max_len=200, max_tokens=300, seed=3, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [torch.randn(n, k, generator=g, device="cuda") * k ** -0.5 for n, k in (((Hq + 2 * Hkv) * D, hidden), (hidden, Hq * D))]
    qw, kw_ = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")
    return K.AttentionBlock(*K.quantise_weight(w[0]), *K.quantise_weight(w[1]), Hq, Hkv, D, K.rope_table(max_len, D), qw, kw_,
                            max_seqs=max_seqs, max_len=max_len, max_tokens=max_tokens, **kw)


def _x(T, hidden, seed):
    return torch.randn(T, hidden, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def test_quantise_weight():
    """Every value is off by at most half a code: 2^-4 of itself, or 2^-10 of the block's scale; no scale is too small or twice too large."""
    g = np.random.default_rng(1)
    w = np.float32(g.normal(0, 1, (300, 200)) * np.exp(g.normal(0, 2, (300, 1))))
    w[130:256, :128] = 0
    codes, scale = K.quantise_weight(_gpu(w))
    c = R.E4M3[codes.view(torch.uint8).cpu().numpy()]
    s = np.exp2(scale.cpu().numpy().astype(np.float64) - 127)
    full = np.repeat(np.repeat(s, 128, 0), 128, 1)[:300, :200]
    assert np.all(np.abs(c * full - w) <= np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10 * full))
    for i in range(3):
        for j in range(2):
            top = np.abs(w[128 * i:128 * i + 128, 128 * j:128 * j + 128]).max()
            assert top <= 448 * s[i, j] and (2 * top > 448 * s[i, j] or top < 2.0 ** -90)


def test_prompt_equals_the_operators_by_hand():
    b = _block()
    print("[block] prompt", flush=True)
    lens = [70, 0, 1, 129]
    x = _x(200, 272, 1)
    p = b.plan(lens)
    y = b.forward(x, p).clone()
    qkv = A.fp8_linear(x, b.w_qkv, b.qkv_scale).view(200, 12, 64)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    q, k = A.qk_norm_rope(qkv[:, :8], qkv[:, 8:10], b.q_weight, b.k_weight, pos, b.cos_sin)
    cu = torch.tensor([0, 70, 70, 71, 200], dtype=torch.int32, device="cuda")
    o = A.attention(q, k, qkv[:, 10:], cu, 129)
    assert torch.equal(b.o[:200], o)
    assert torch.equal(y, A.fp8_linear(o.view(200, 512), b.w_out, b.out_scale))
    for s, (a, n) in enumerate(zip([0, 70, 70, 71], lens)):
        assert torch.equal(b.cache[200 * s:200 * s + n, :2], k[a:a + n])
        assert torch.equal(b.cache[200 * s:200 * s + n, 2:], qkv[a:a + n, 10:])


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (4, 1, 256)])
def test_chunks_and_single_tokens(Hq, Hkv, D):
    """A prompt in chunks of any size, a mixture of chunks and single tokens, then single tokens with an advanced plan:
    after each call the attention and the projection against the references, over what the cache then holds."""
    b = _block(Hq, Hkv, D, seed=D)
    lens = np.zeros(4, int)
    step = None
    calls = [[40, 1, 0, 17], [3, 1, 5, 1], [0, 90, 1, 1], [1, 1, 1, 1], None, None]
    for i, new in enumerate(calls):
        print("[block] call", Hq, Hkv, D, new, flush=True)
        if new is None:
            step.advance()
            new = [1, 1, 1, 1]
        else:
            step = b.plan(new, max_kv=200 if i == 3 else None)
        lens += new
        T = sum(new)
        x = _x(T, 272, 10 + i)
        y = b.forward(x, step)
        cu = np.r_[0, np.cumsum(new)]
        seqs = [(int(cu[s]), new[s], 200 * s, int(lens[s])) for s in range(4)]
        assert step.kv_len.tolist() == lens.tolist()
        kv = _np(b.cache)
        for q0, n, k0, m in seqs:  # rows past a sequence's end hold whatever the allocation held
            kv[k0 + m:k0 + 200] = 0
        # the queries as the block holds them after norm and rotation
        _check_attention(b.o[:T], None, _np(b.qkv[:T, :Hq]), kv[:, :Hkv], kv[:, Hkv:], seqs, D ** -0.5, True)
        for s, (q0, n, k0, m) in enumerate(seqs):
            assert torch.equal(b.cache[k0 + m - n:k0 + m], b.qkv[q0:q0 + n, Hq:])
        codes, sc = b.w_out.view(torch.uint8).cpu().numpy(), np.exp2(b.out_scale.cpu().numpy().astype(np.float64) - 127)
        ref, mag, top = R.fp8_linear(_np(b.o[:T].reshape(T, -1)), codes, sc, "e8m0")
        _check_linear(y, ref, mag, top, Hq * D)


def test_refusals():
    b = _block(max_seqs=2, max_len=20, max_tokens=30)
    print("[block] refusals", flush=True)
    for new in ([1, 1, 1], [-1], [21], [20, 20]):
        with pytest.raises(ValueError):
            b.plan(new)
    assert b.lens == [0, 0]
    p = b.plan([20, 3])
    with pytest.raises(ValueError):
        b.plan([1, 0])
    assert b.lens == [20, 3]
    with pytest.raises(ValueError):
        b.forward(_x(22, 272, 0), p)
    with pytest.raises(ValueError):
        b.forward(_x(23, 256, 0), p)
    with pytest.raises(ValueError):
        K.AttentionBlock(b.w_qkv, b.qkv_scale, b.w_out, b.out_scale, 8, 3, 64, b.cos_sin, max_seqs=1, max_len=8, max_tokens=8)
    with pytest.raises(ValueError):
        K.AttentionBlock(b.w_qkv, b.qkv_scale, b.w_qkv, b.qkv_scale, 8, 2, 64, b.cos_sin, max_seqs=1, max_len=8, max_tokens=8)
    with pytest.raises(ValueError):
        K.AttentionBlock(b.w_qkv, b.qkv_scale, b.w_out, b.out_scale, 8, 2, 64, b.cos_sin, max_seqs=1, max_len=21, max_tokens=8)


def test_example_eager_and_graph():
    print("[block] example", flush=True)
    eager, replayed = K.example()
    assert len(eager) == len(replayed) == 6
    for a, b in zip(eager, replayed):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_a_plan_after_advances_and_their_bounds():
    """What advances and replays brought counts for later plans; a plan stops at its bound, and a bound at the cache's room."""
    b = _block(max_seqs=3, max_len=20, max_tokens=30)
    print("[block] advances", flush=True)
    prompt = b.plan([5, 0, 9])
    b.forward(_x(14, 272, 1), prompt)
    with pytest.raises(ValueError):
        prompt.advance()
    for bound in (9, 21):
        with pytest.raises(ValueError):
            b.plan([1, 0, 1], max_kv=bound)
    assert b.lens == [5, 0, 9]
    step = b.plan([1, 0, 1], max_kv=12)
    for i in range(3):
        b.forward(_x(2, 272, 2 + i), step)
        step.advance()
    with pytest.raises(ValueError):
        b.forward(_x(2, 272, 5), step)
    assert b.lens == [9, 0, 13] and step.kv_len.tolist() == [9, 3, 13]
    b.lens[:] = [8, 0, 12]  # the step that was refused
    late = b.plan([2, 4, 1])
    x = _x(7, 272, 6)
    b.forward(x, late)
    assert late.positions.tolist() == [8, 9, 0, 1, 2, 3, 12] and late.kv_len.tolist() == [10, 4, 13]
    seqs = [(0, 2, 0, 10), (2, 4, 20, 4), (6, 1, 40, 13)]
    kv = _np(b.cache)
    kv[10:20], kv[24:40], kv[53:] = 0, 0, 0
    _check_attention(b.o[:7], None, _np(b.qkv[:7, :8]), kv[:, :2], kv[:, 2:], seqs, 64 ** -0.5, True)
    one = b.plan([1], max_kv=20)
    one.replayed(4)
    assert b.lens[0] == 15 and one.longest == 15


@pytest.mark.parametrize("graph", [False, True])
def test_chunks_after_the_step_loop(graph):
    """forward, advance, forward, advance, ... eager or as a graph of both, then a chunk: its attention is that of the
    reference over every token that ran, and over no row that none wrote."""
    b = _block(max_seqs=3, max_len=40, max_tokens=30)
    print("[block] chunk after the loop", graph, flush=True)
    b.cache.fill_(float("nan"))
    b.forward(_x(14, 272, 1), b.plan([5, 0, 9]))
    step = b.plan([1, 0, 1], max_kv=30)
    x = _x(2, 272, 2)
    if graph:
        start = [t.clone() for t in (step.positions, step.kv_len, step.rows)]
        ws = b.workspace(step)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.forward(x, step, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.forward(x, step, ws)
            step.advance()
        for t, v in zip((step.positions, step.kv_len, step.rows), start):
            t.copy_(v)
        step.replayed(3)
        for _ in range(4):
            g.replay()
    else:
        for _ in range(4):
            b.forward(x, step)
            step.advance()
    torch.cuda.synchronize()
    assert [b.held(s) for s in range(3)] == [9, 0, 13]
    late = b.plan([2, 4, 1])
    b.forward(_x(7, 272, 6), late)
    assert late.positions.tolist() == [9, 10, 0, 1, 2, 3, 13] and late.kv_len.tolist() == [11, 4, 14]
    kv = _np(b.cache)
    for s, n in enumerate((11, 4, 14)):
        assert np.isfinite(kv[40 * s:40 * s + n]).all() and np.isnan(kv[40 * s + n:40 * s + 40]).all()
    seqs = [(0, 2, 0, 11), (2, 4, 40, 4), (6, 1, 80, 14)]
    _check_attention(b.o[:7], None, _np(b.qkv[:7, :8]), np.nan_to_num(kv[:, :2]), np.nan_to_num(kv[:, 2:]), seqs, 64 ** -0.5, True)


def test_replays_past_the_end_of_the_cache():
    """A graph of forward and advance() replayed more often than there is room: the other sequences' rows keep their bits."""
    b = _block(max_seqs=3, max_len=20, max_tokens=30)
    print("[block] replays past the end", flush=True)
    b.forward(_x(25, 272, 1), b.plan([4, 18, 3]))
    step = b.plan([0, 1, 1], max_kv=20)
    x, ws = _x(2, 272, 2), b.workspace(step)
    start = [t.clone() for t in (step.positions, step.kv_len, step.rows)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward(x, step, ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.forward(x, step, ws)
        step.advance()
    for t, v in zip((step.positions, step.kv_len, step.rows), start):
        t.copy_(v)
    with pytest.raises(ValueError):
        step.replayed(2)
    step.replayed(1)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    held = b.cache.view(torch.int16).clone()
    assert step.kv_len.tolist() == [6, 21, 6] and step.rows.tolist() == [39, 45]
    for _ in range(30):
        g.replay()
    torch.cuda.synchronize()
    now = b.cache.view(torch.int16)
    assert step.rows.tolist() == [39, 59]
    for lo, hi in ((0, 39), (40, 45)):
        assert torch.equal(now[lo:hi], held[lo:hi])


def test_a_plan_of_no_tokens():
    b = _block()
    print("[block] no tokens", flush=True)
    for new in ([], [0, 0]):
        plan = b.plan(new)
        assert b.forward(_x(0, 272, 1), plan, b.workspace(plan)).shape == (0, 272)
    assert b.lens == [0, 0, 0, 0]
