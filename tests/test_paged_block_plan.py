"""The bookkeeping of PagedAttentionBlock on the CPU: stand-ins for the operators carry a token's number from x
to its slot, and every call is checked for what its attention reads through the page table: token j of a
sequence at position j, none missing, the same through the group's first sequence for what a group shares."""
import random

import pytest

torch = pytest.importorskip("torch")

from mxfp4_routed_expert_moe_amd import block as K  # noqa: E402

HQ, HKV, D, HIDDEN = 2, 1, 8, 32


class Model:
    """A block and what was fed to it."""

    def __init__(self, monkeypatch, max_seqs=4, max_len=200, max_tokens=300, n_pages=40, page_size=16, select=None):
        self.calls = []

        def linear(x, w, scale, y=None, ws=None):
            y[:] = x[:, :1]
            return y

        def append(k, v, k_pages, v_pages, cu_q, kv_len, table, **kw):
            for b in range(len(kv_len)):
                n = int(cu_q[b + 1] - cu_q[b])
                for i in range(n):
                    p = int(kv_len[b]) - n + i
                    page = int(table[b, p // page_size]) if p // page_size < table.shape[1] else -1
                    if page >= 0:
                        k_pages[page, p % page_size] = k[cu_q[b] + i]
            return kw["q_out"]

        def attention(q, k_pages, v_pages, cu_q, kv_len, table, max_q, max_kv, *, cu_group=None, prefix_len=None, max_prefix=0,
                      blocks=None, out=None, ws=None):
            self.calls.append((cu_q.tolist(), kv_len.tolist(), table.clone(), max_q, max_kv,
                               None if cu_group is None else (cu_group.tolist(), prefix_len.tolist(), max_prefix), blocks))
            out.zero_()
            return out

        def pick(q, bounds, cu_q, kv_len, table, max_q, max_kv, size, n, *, first, last, blocks, ws=None):
            assert (size, n, first, last) == (page_size, *select)
            blocks.zero_()
            return blocks

        monkeypatch.setattr(K.A, "fp8_linear", linear)
        for name, f in (("paged_append", append), ("paged_attention", attention), ("select_blocks", pick)):
            monkeypatch.setattr(K.P, name, f)
        code = torch.zeros
        self.b = K.PagedAttentionBlock(code((HQ + 2 * HKV) * D, HIDDEN), None, code(HIDDEN, HQ * D), None, HQ, HKV, D,
                                       torch.zeros(max_len, D), max_seqs=max_seqs, max_len=max_len, max_tokens=max_tokens,
                                       n_pages=n_pages, page_size=page_size, select=select)
        self.b.cache.fill_(float("nan"))  # a slot that was never written
        self.size = page_size
        self.fed = [[] for _ in range(max_seqs)]
        self.next = 1

    def x(self, new):
        """Tokens with the next numbers, noted per sequence."""
        tokens = []
        for s, n in enumerate(new):
            for _ in range(n):
                self.fed[s].append(self.next)
                tokens.append(self.next)
                self.next = self.next % 200 + 1  # numbers that bf16 holds
        return torch.tensor(tokens).float()[:, None].expand(len(tokens), HIDDEN).bfloat16()

    def read(self, table_row, n):
        k = self.b.cache[:, :, 0, 0]
        return [float(k[int(table_row[p // self.size]), p % self.size]) for p in range(n)]

    def step(self, new, plan=None):
        """Runs a plan and checks what its attention saw.  -> the plan"""
        plan = plan or self.b.plan(new)
        self.b.forward(self.x(new), plan)
        cu, length, table, max_q, max_kv, group, blocks = self.calls[-1]
        of = {}
        if group:
            bounds, prefix, most = group
            for i, j, p in zip(bounds, bounds[1:], prefix):
                assert p <= most and p % self.size == 0
                for s in range(i, j):
                    of[s] = (i, p)
        for s, n in enumerate(new):
            assert cu[s + 1] - cu[s] == n <= max_q
            if not n:
                continue
            first, p = of.get(s, (s, 0))
            assert length[s] == len(self.fed[s]) and length[s] - p <= max_kv
            assert self.read(table[s], length[s]) == [float(t) for t in self.fed[s]]
            assert self.read(table[first], p) == [float(t) for t in self.fed[s][:p]]
        return plan

    def check_pages(self):
        """Every page is free or held, and counted once per sequence that holds it."""
        held = [p for pages in self.b.pages for p in pages]
        assert sorted(set(held) | set(self.b.free)) == list(range(self.b.n_pages)) and not set(held) & set(self.b.free)
        assert len(set(self.b.free)) == len(self.b.free)
        assert all(self.b.users[p] == held.count(p) for p in range(self.b.n_pages))
        for s, pages in enumerate(self.b.pages):
            assert self.b.table[s, :len(pages)].tolist() == pages and torch.all(self.b.table[s, len(pages):] == -1)

    def fork(self, src, dst):
        self.b.fork(src, dst)
        self.fed[dst] = list(self.fed[src])
        self.check_pages()


def test_prompts_chunks_and_steps(monkeypatch):
    m = Model(monkeypatch)
    for new in ([40, 0, 7, 1], [3, 20, 0, 16], [1, 1, 1, 1], [0, 0, 30, 0]):
        m.step(new)
        m.check_pages()
    assert [len(p) for p in m.b.pages] == [3, 2, 3, 2]


def test_forks_share_what_is_full(monkeypatch):
    m = Model(monkeypatch)
    m.step([50])
    m.fork(0, 2)
    m.fork(2, 1)
    assert m.b.pages[0][:3] == m.b.pages[1][:3] == m.b.pages[2][:3] and len({p[3] for p in m.b.pages[:3]}) == 3
    m.step([1, 1, 1])
    assert m.calls[-1][5] == ([0, 3], [48], 48)
    m.step([3, 0, 20])  # an idle one between
    assert m.calls[-1][5] == ([0, 3], [48], 48)
    m.step([0, 1, 0, 5])
    assert m.calls[-1][5] is None  # nobody shares with a neighbour that brings rows
    m.step([0, 1, 1, 1])
    assert m.calls[-1][5] == ([1, 3, 4], [48, 0], 48)
    m.b.reset(0)
    m.fed[0] = []
    m.check_pages()
    m.step([5, 1, 1])
    m.b.reset()
    assert sorted(m.b.free) == list(range(40)) and not any(m.b.users)


def test_fork_at_a_page_end_and_of_nothing(monkeypatch):
    m = Model(monkeypatch)
    m.fork(0, 1)
    assert m.b.pages[1] == []
    m.step([32, 1])
    m.fork(0, 3)
    assert m.b.pages[3] == m.b.pages[0]
    m.step([1, 0, 0, 1])
    assert m.b.pages[3][:2] == m.b.pages[0][:2] and m.b.pages[3][2] != m.b.pages[0][2]


def test_groups_join_while_they_share_enough(monkeypatch):
    """A long shared prefix is not given up for a neighbour that shares little."""
    m = Model(monkeypatch)
    m.step([20])
    m.fork(0, 3)          # shares one page with the others
    m.step([140])
    m.fork(0, 1)
    m.fork(0, 2)          # shares ten
    m.step([1, 1, 1, 1])
    assert m.calls[-1][5] == ([0, 3, 4], [160, 0], 160)


def test_advanced_plans_have_their_pages(monkeypatch):
    m = Model(monkeypatch)
    m.step([30, 15])
    plan = m.b.plan([1, 1], max_kv=70)
    assert [len(p) for p in m.b.pages[:2]] == [5, 4]  # 70 and 55 tokens
    for i in range(40):
        m.step([1, 1], plan)
        if i < 39:
            plan.advance()
    m.check_pages()
    assert [len(f) for f in m.fed[:2]] == [70, 55]
    with pytest.raises(ValueError):
        plan.advance()
        m.b.forward(m.x([1, 1]), plan)


def test_refusals(monkeypatch):
    m = Model(monkeypatch, n_pages=6)
    plan = m.step([60])
    for bad in ((0, 0), (0, 4), (-1, 1), (4, 0)):
        with pytest.raises(ValueError):
            m.b.fork(*bad)
    with pytest.raises(ValueError):
        m.b.plan([0, 33])  # three pages, two are free
    m.check_pages()
    assert m.b.lens == [60, 0, 0, 0]
    m.fork(0, 1)
    m.step([0, 1])
    with pytest.raises(ValueError):
        m.b.fork(0, 1)  # holds tokens
    late = m.b.plan([1])
    with pytest.raises(ValueError):
        m.b.fork(0, 2)  # a plan has not run
    late.cancel()
    m.b.reset(1)
    m.step([0, 0, 32])
    with pytest.raises(ValueError):
        m.b.fork(0, 3)  # no page for the last one's copy
    m.check_pages()
    m.b.reset(0)
    m.check_pages()
    with pytest.raises(ValueError):
        m.b.forward(m.x([60]), plan)
    for kw in (dict(page_size=24), dict(n_pages=0), dict(select=(2, 1, 2)), dict(select=(4, 1, 0)), dict(select=(2000, 1, 1))):
        with pytest.raises(ValueError):
            Model(monkeypatch, **kw)


def test_selection_is_for_single_tokens(monkeypatch):
    m = Model(monkeypatch, select=(4, 1, 2))
    m.step([100, 30])
    assert m.calls[-1][6] is None
    m.step([1, 1])
    assert m.calls[-1][6].shape == (2, HKV, 4)
    m.step([2, 1])
    assert m.calls[-1][6] is None
    m.fork(0, 2)
    m.step([1, 0, 1])
    assert m.calls[-1][6] is not None and m.calls[-1][5] is None


def test_empty_plan(monkeypatch):
    m = Model(monkeypatch)
    plan = m.b.plan([])
    assert m.b.forward(torch.zeros(0, HIDDEN).bfloat16(), plan).shape == (0, HIDDEN)
    m.check_pages()


def test_a_plan_does_not_run_again_over_shared_pages(monkeypatch):
    """What a fork shares is written no more: a plan of the sequence that ran before is refused as long as another one holds a
    page of its rows, and what its replay would store stays out of them."""
    m = Model(monkeypatch)
    first = m.step([40])
    more = m.step([3])
    again = m.x([40])
    m.fed[0] = m.fed[0][-40:] + m.fed[0][40:43]  # the first plan runs anew: no fork yet
    m.b.forward(again, first)
    assert m.read(m.b.table[0], 43) == [float(t) for t in m.fed[0]]
    m.fork(0, 1)
    kept = m.read(m.b.table[1], 43)
    with pytest.raises(ValueError):
        m.b.forward(m.x([40]), first)
    m.b._enqueue(torch.full((40, HIDDEN), 7.0).bfloat16(), first, None)  # as a replay of a graph, which no check sees
    assert m.read(m.b.table[1], 43) == kept and m.read(m.b.table[0], 32) == kept[:32]
    m.fed[0] = m.fed[1] + []
    m.b._enqueue(torch.tensor(m.fed[0][:40]).float()[:, None].expand(40, HIDDEN).bfloat16(), first, None)
    m.b.forward(torch.tensor(m.fed[0][40:]).float()[:, None].expand(3, HIDDEN).bfloat16(), more)  # in a page of its own
    m.step([2, 1])
    m.fork(1, 2)
    m.b.reset(1)
    m.fed[1] = []
    m.check_pages()
    with pytest.raises(ValueError):
        m.b.forward(m.x([40]), first)  # sequence 2 still holds the pages
    m.fed[0] = m.fed[0][:45]
    m.b.reset(2)
    m.fed[2] = []
    tokens = m.fed[0][:40]
    m.b.forward(torch.tensor(tokens[::-1]).float()[:, None].expand(40, HIDDEN).bfloat16(), first)  # alone again
    assert m.read(m.b.table[0], 40) == [float(t) for t in tokens[::-1]]


def test_a_step_does_not_run_again_into_a_page_that_it_filled(monkeypatch):
    m = Model(monkeypatch)
    m.step([31, 5])
    step = m.b.plan([1, 1], max_kv=40)
    m.step([1, 1], step)
    m.fork(0, 2)
    with pytest.raises(ValueError):
        m.b.forward(m.x([1, 1]), step)  # token 31 of sequence 0 is in a page that sequence 2 holds
    m.fed = [f[:n] for f, n in zip(m.fed, (32, 6, 32, 0))]
    step.advance()
    m.step([1, 1], step)  # the next one is in a page of its own
    m.step([0, 0, 4])
    m.check_pages()


def test_the_tables_name_pages_and_what_may_be_written(monkeypatch):
    """After forks and resets in any order the device tables are what the host knows."""
    m = Model(monkeypatch, n_pages=30)

    def check():
        m.check_pages()
        for s, pages in enumerate(m.b.pages):
            own = [p if m.b.users[p] == 1 else -1 for p in pages]
            assert m.b.own[s].tolist() == own + [-1] * (m.b.own.shape[1] - len(own))

    m.step([50])
    for do in ((m.fork, 0, 2), (m.fork, 2, 1), (m.step, [1, 20, 1]), (m.b.reset, 2), (m.fork, 1, 3), (m.b.reset, 0), (m.b.reset, 3),
               (m.fork, 1, 0), (m.b.reset,)):
        do[0](*do[1:])
        if do[0] == m.b.reset:
            for s in range(4) if len(do) == 1 else do[1:]:
                m.fed[s] = []
        check()


def test_cancelled_plans_give_their_pages_back(monkeypatch):
    """Those that no token of the sequence's other plans needs: also the ones kept for steps of an advanced plan, and not
    those of a plan that has yet to run, or shared ones."""
    m = Model(monkeypatch, n_pages=10)
    plan = m.b.plan([150])
    assert not m.b.free
    plan.cancel()
    m.check_pages()
    assert m.b.pages[0] == []
    m.step([20, 20])  # the pages are there again
    steps = m.b.plan([1, 1], max_kv=60)
    assert [len(p) for p in m.b.pages] == [4, 4, 0, 0]
    steps.cancel()
    m.check_pages()
    assert [len(p) for p in m.b.pages] == [2, 2, 0, 0]
    first, second = m.b.plan([20]), m.b.plan([50])
    assert len(m.b.pages[0]) == 6
    second.cancel()
    m.check_pages()
    assert len(m.b.pages[0]) == 3  # 40 tokens, 20 of them in the plan that runs now
    m.step([20], first)
    m.fork(0, 2)
    plan = m.b.plan([0, 10, 40])
    m.b.reset(1)
    m.fed[1] = []
    plan.cancel()
    m.check_pages()
    assert [len(p) for p in m.b.pages] == [3, 0, 3, 0] and m.b.pages[2][:2] == m.b.pages[0][:2]
    m.step([1, 0, 1])
    m.fork(1, 3)


def test_a_cancelled_step_gives_back_what_was_kept_for_it(monkeypatch):
    """An advanced plan ends with a plan behind it, so a cancel of that one leaves the sequence what its tokens need."""
    m = Model(monkeypatch, n_pages=8)
    m.step([15])
    step = m.b.plan([1], max_kv=100)
    for i in range(3):
        m.step([1], step)
        if i < 2:
            step.advance()
    assert len(m.b.pages[0]) == 7
    m.b.plan([2]).cancel()
    m.check_pages()
    assert len(m.b.pages[0]) == 2
    with pytest.raises(ValueError):
        step.advance()
    m.step([100])
    m.check_pages()


def test_selection_past_its_limits_is_refused_with_the_plan(monkeypatch):
    """More blocks than the choice can rank: the plan is refused before it takes pages, not its run after the append."""
    m = Model(monkeypatch, max_len=32768 * 16 + 100, n_pages=64, select=(4, 1, 2))
    m.step([100, 30])
    for bound in (32768 * 16 + 1, 32768 * 16 + 100):
        with pytest.raises(ValueError, match="32768"):
            m.b.plan([1, 1], max_kv=bound)
        with pytest.raises(ValueError, match="free"):
            m.b.plan([1, 1], max_kv=bound - 101)  # not past the limit: refused for want of pages
    m.check_pages()
    m.step([1, 1], m.b.plan([1, 1], max_kv=200))
    m.step([2, 1], m.b.plan([2, 1], max_kv=32768 * 16 + 100))  # selects nothing
    m.check_pages()


def test_selecting_plans_have_no_groups(monkeypatch):
    """Every sequence's chosen pages are read for itself: nothing is made for groups that no call reads."""
    m = Model(monkeypatch, select=(4, 1, 2))
    m.step([100])
    m.fork(0, 1)
    assert m.b.plan([1, 1]).group is None
    m.b.reset()
    m.fed = [[] for _ in m.fed]
    m.step([100])
    m.fork(0, 1)
    m.step([2, 1])
    assert m.calls[-1][5] == ([0, 2], [96], 96)


@pytest.mark.parametrize("seed", range(50))
def test_random_walks(monkeypatch, seed):
    """Plans, steps, cancels, forks, resets and second runs in any order: what a sequence reads is what it was fed, whatever the others
    do, and every page is accounted for."""
    r = random.Random(seed)
    m = Model(monkeypatch, n_pages=r.choice([14, 24, 40]), max_len=160, select=r.choice([None, (4, 1, 2)]))
    ran = []  # plans that have run, and how many tokens there were before
    for _ in range(60):
        do = r.choice(["step", "step", "decode", "cancel", "fork", "fork", "reset", "again", "again"])
        held = [len(f) for f in m.fed]
        new = [r.choice([0, 0, 0, 1, 5, 17, 40]) for _ in held]
        new[r.randrange(4)] = r.choice([1, 30])
        try:
            if do == "step":
                plan = m.b.plan(new)
                m.step(new, plan)
                ran.append((plan, held))
            elif do == "decode":
                who = [int(h > 0 and r.random() < 0.7) for h in held]
                who[r.randrange(4)] = 1
                plan = m.b.plan(who, max_kv=min(160, max(h + 1 for h, w in zip(held, who) if w) + r.randint(0, 20)))
                for i in range(r.randint(1, min(5, plan.max_kv - plan.longest + 1))):
                    if i:
                        plan.advance()
                    m.step(who, plan)
            elif do == "cancel":
                plan, other = m.b.plan(new), r.random() < 0.5
                if other:
                    m.b.plan([1] * 4).cancel()
                plan.cancel()
            elif do == "fork":
                m.fork(r.randrange(4), r.randrange(4))
            elif do == "reset":
                b = r.randrange(4)
                m.b.reset(b)
                m.fed[b] = []
            elif ran:
                plan, at = r.choice(ran)
                tokens = [r.randint(1, 200) for _ in range(sum(plan.new))]  # other ones in the same places
                m.b.forward(torch.tensor(tokens).float()[:, None].expand(len(tokens), HIDDEN).bfloat16(), plan)
                for s, n in enumerate(plan.new):
                    m.fed[s][at[s]:at[s] + n], tokens = tokens[:n], tokens[n:]
        except ValueError:
            for plan in m.b._unrun:
                assert len(plan) <= 1
            for s in range(4):  # a plan that did not get to run
                if m.b._unrun[s]:
                    m.b.reset(s)
                    m.fed[s] = []
        m.check_pages()
        for s, f in enumerate(m.fed):
            assert m.b.held(s) == len(f)
            assert m.read(m.b.table[s], len(f)) == [float(t) for t in f]
