"""The bookkeeping of AttentionBlock on the CPU: stand-ins for the operators carry a
token's number from x to its cache row, and every call is checked for the rows that
its attention reads: token j of a sequence in row j, at position j, none missing."""
import pytest

torch = pytest.importorskip("torch")

from mxfp4_routed_expert_moe_amd import block as K  # noqa: E402

HQ, HKV, D, HIDDEN = 2, 1, 8, 32


class Model:
    """A block and what was fed to it."""

    def __init__(self, monkeypatch, max_seqs=3, max_len=20, max_tokens=30):
        self.calls = []

        def linear(x, w, scale, y=None, ws=None):
            y[:] = x[:, :1]
            return y

        def rope(q, k, qw, kw, positions, cos_sin, **kw_):
            self.positions = positions.clone()
            return q, k

        def attention(q, k, v, cu_q, max_q, *, kv_start, kv_len, max_kv, out, ws=None):
            self.calls.append((cu_q.tolist(), kv_start.tolist(), kv_len.tolist(), max_q, max_kv))
            out.zero_()
            return out

        for name, f in (("fp8_linear", linear), ("qk_norm_rope", rope), ("attention", attention)):
            monkeypatch.setattr(K.A, name, f)
        code = torch.zeros
        self.b = K.AttentionBlock(code((HQ + 2 * HKV) * D, HIDDEN), None, code(HIDDEN, HQ * D), None, HQ, HKV, D,
                                  torch.zeros(max_len, D), max_seqs=max_seqs, max_len=max_len, max_tokens=max_tokens)
        self.b.cache.fill_(float("nan"))  # a row that was never written
        self.fed = [[] for _ in range(max_seqs)]
        self.next = 1

    def x(self, new):
        """Tokens with the next numbers, noted per sequence."""
        T = sum(new)
        for s, n in enumerate(new):
            self.fed[s] += range(self.next, self.next + n)
            self.next += n
        return torch.arange(self.next - T, self.next).float()[:, None].expand(T, HIDDEN).bfloat16()

    def check(self, new):
        """The last call read, for each of its sequences, every token fed so far and nothing else."""
        cu, start, length, max_q, max_kv = self.calls[-1]
        at = 0
        for s, n in enumerate(new):
            assert cu[s + 1] - cu[s] == n <= max_q
            if n == 0:
                continue
            have = len(self.fed[s])
            assert length[s] == have <= max_kv
            assert self.b.cache[start[s]:start[s] + have, 0, 0].tolist() == self.fed[s]
            assert self.positions[at:at + n].tolist() == list(range(have - n, have))
            at += n

    def run(self, new, plan=None, **kw):
        plan = plan or self.b.plan(new, **kw)
        self.b.forward(self.x(new), plan)
        self.check(new)
        return plan

    def replay(self, plan):
        """What a HIP graph of forward and advance() does: the device's part alone."""
        x = self.x(plan.new)
        self.b._enqueue(x, plan, None)
        self.check(plan.new)
        plan._shift()


@pytest.fixture
def model(monkeypatch):
    return Model(monkeypatch)


@pytest.mark.parametrize("steps", [1, 3])
@pytest.mark.parametrize("last", [True, False])
def test_a_plan_after_forward_and_advance(model, steps, last):
    """forward, advance, forward, advance, ...: whether or not the loop ends with an advance, the next plan's tokens
    follow those that ran."""
    model.run([5, 0, 9])
    step = model.b.plan([1, 0, 1], max_kv=20)
    for i in range(steps):
        model.run([1, 0, 1], step)
        if i + 1 < steps or last:
            step.advance()
    model.run([2, 4, 1])
    model.run([1, 1, 1])


def test_a_plan_beside_an_announced_step(model):
    """A plan that brings nothing to a sequence leaves the step that was announced for it in place."""
    model.run([5, 2])
    step = model.run([1], max_kv=20)
    step.advance()
    model.run([0, 3])
    model.run([1], step)
    step.advance()
    model.run([1], step)
    model.run([2, 1])


def test_plans_made_ahead(model):
    """Plans are made in the order in which they run, and may be made before."""
    plans = [([3, 4], model.b.plan([3, 4])), ([2, 0], model.b.plan([2, 0])), ([1, 1], model.b.plan([1, 1], max_kv=20))]
    for i, (new, plan) in enumerate(plans):
        model.b.forward(model.x(new), plan)
        if i != 1:
            model.check(new)
    plans[-1][1].advance()
    model.run([1, 1], plans[-1][1])


def test_a_step_whose_place_was_taken(model):
    """A plan that brings tokens to a sequence takes the place of a step announced for it: that one is refused."""
    model.run([5])
    step = model.run([1], max_kv=20)
    step.advance()
    model.run([2])
    for f in (lambda: model.b.forward(torch.zeros(1, HIDDEN).bfloat16(), step), step.advance, lambda: step.replayed(2)):
        with pytest.raises(ValueError):
            f()
    model.run([1])


@pytest.mark.parametrize("replays", [1, 4])
def test_a_plan_after_graph_replays(model, replays):
    """The example's use: one step outside the graph, capture of forward and advance (counts the first replay), the
    state put back, replays, replayed() for the others."""
    model.run([5, 0, 9])
    step = model.b.plan([1, 0, 1], max_kv=20)
    state = [t.clone() for t in (step.positions, step.kv_len, step.rows)]
    zeros = torch.zeros(2, HIDDEN).bfloat16()
    model.b.forward(zeros, step)
    model.b.forward(zeros, step)
    step.advance()
    for t, v in zip((step.positions, step.kv_len, step.rows), state):
        t.copy_(v)
    step.replayed(replays - 1)
    for _ in range(replays):
        model.replay(step)
    model.run([3, 2, 1])


def test_a_graph_of_forward_alone(model):
    """advance() outside the graph: each counts the replay before it."""
    model.run([4])
    step = model.b.plan([1], max_kv=20)
    model.b.forward(torch.zeros(1, HIDDEN).bfloat16(), step)  # the capture
    for _ in range(3):
        model.b._enqueue(model.x([1]), step, None)
        model.check([1])
        step.advance()
    model.run([2])


def test_a_full_sequence_and_its_slot(model):
    """A sequence filled to the cache's end by a loop that ends with an advance: plans beside it go on, more tokens for it
    are refused, and reset makes its slot free for another sequence."""
    model.run([18, 2])
    step = model.b.plan([1], max_kv=20)
    for _ in range(2):
        model.run([1], step)
        step.advance()
    with pytest.raises(ValueError):
        model.b.forward(torch.zeros(1, HIDDEN).bfloat16(), step)
    model.run([0, 3])
    with pytest.raises(ValueError):
        model.b.plan([1])
    model.b.reset(0)
    model.fed[0] = []
    with pytest.raises(ValueError):
        step.advance()
    model.run([4, 1])
    model.b.reset()
    model.fed = [[], [], []]
    model.run([1, 2, 20])
    for bad in (-1, 3):
        with pytest.raises(ValueError):
            model.b.reset(bad)


def test_reset_of_a_sequence_with_an_announced_step(model):
    model.run([3, 4])
    step = model.run([1, 1], max_kv=20)
    step.advance()
    model.b.reset(1)
    model.fed[1] = []
    with pytest.raises(ValueError):
        model.b.forward(torch.zeros(2, HIDDEN).bfloat16(), step)
    model.run([2, 2])


@pytest.mark.parametrize("lens", [[15, 5], [20, 0]])
def test_a_long_idle_sequence_does_not_bound_the_others(model, lens):
    """max_kv bounds the sequences that a plan brings tokens to; an idle one beside them may be longer, or full."""
    model.run(lens)
    bound = lens[1] + 3
    with pytest.raises(ValueError):
        model.b.plan([0, 1], max_kv=lens[1])
    step = model.b.plan([0, 1], max_kv=bound)
    for _ in range(3):
        model.run([0, 1], step)
        assert model.calls[-1][-1] == bound
        step.advance()
    with pytest.raises(ValueError):
        model.b.forward(torch.zeros(1, HIDDEN).bfloat16(), step)
    plan = model.b.plan([0, 2])
    assert plan.max_kv == lens[1] + 5
    model.run([0, 2], plan)


def test_replays_past_the_bound(model):
    """replayed refuses, before the replays, those that would pass max_kv, and changes nothing; replays that were never
    noted stay inside their sequence's rows."""
    model.run([4, 18, 3])
    step = model.b.plan([0, 1, 1], max_kv=20)
    before = list(model.b.lens), step.longest
    for n in (3, -1):
        with pytest.raises(ValueError):
            step.replayed(n)
    assert (list(model.b.lens), step.longest) == before
    step.replayed(2)
    for _ in range(2):
        model.replay(step)
    for f in (step.advance, lambda: step.replayed(1)):
        with pytest.raises(ValueError):
            f()
    cache = model.b.cache.clone()
    for _ in range(30):  # 28 past the end of sequence 1, 13 past that of sequence 2, the last of the cache
        model.b._enqueue(torch.full((2, HIDDEN), 99.0).bfloat16(), step, None)
        step._shift()
    # sequence 0, and all that sequences 1 and 2 hold but the last row of each
    assert torch.equal(model.b.cache[:20].nan_to_num(), cache[:20].nan_to_num())
    assert torch.equal(model.b.cache[20:39], cache[20:39]) and torch.equal(model.b.cache[40:45], cache[40:45])


@pytest.mark.parametrize("new", [[], [0], [0, 0, 0]])
def test_a_plan_of_no_tokens(model, new):
    model.run([3, 1])
    plan = model.b.plan(new)
    calls = len(model.calls)
    assert model.b.forward(torch.empty(0, HIDDEN).bfloat16(), plan).shape == (0, HIDDEN)
    plan.advance()
    assert len(model.calls) == calls
    with pytest.raises(ValueError):
        model.b.forward(torch.empty(1, HIDDEN).bfloat16(), plan)
    model.run([1, 1, 1])


def test_a_plan_that_never_ran(model):
    """Its tokens lie before those of later plans: these are refused until it has run, or gave its tokens back."""
    model.run([3, 4, 1])
    lost = model.b.plan([2, 0, 1])
    other = model.b.plan([0, 2])
    after = model.b.plan([1, 1], max_kv=20)
    with pytest.raises(ValueError):
        model.b.forward(torch.zeros(2, HIDDEN).bfloat16(), after)
    with pytest.raises(ValueError):
        after.replayed(1)
    with pytest.raises(ValueError):  # a later plan goes on from its tokens
        lost.cancel()
    model.run([0, 2], other)
    after.cancel()
    lost.cancel()
    assert model.b.lens == [3, 6, 1]
    for f in (lambda: model.b.forward(torch.zeros(3, HIDDEN).bfloat16(), lost), lost.cancel, after.advance, other.cancel):
        with pytest.raises(ValueError):
            f()
    model.run([2, 1, 1])


def test_reset_forgets_plans_that_never_ran(model):
    lost = model.b.plan([2, 3])
    model.b.reset(0)
    model.run([4])
    with pytest.raises(ValueError):
        model.b.forward(torch.zeros(5, HIDDEN).bfloat16(), lost)
    with pytest.raises(ValueError):
        model.run([1, 1])
    model.b.reset()
    model.fed = [[], [], []]
    model.run([1, 1])
