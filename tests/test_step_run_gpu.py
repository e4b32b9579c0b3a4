"""The operators of a speculative decoding step together, as a serving loop calls them: in
turn, on streams and in captured graphs, on caches past 4 GiB, over random shapes.
Tolerances: tests/test_step_ops_gpu.py."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests import step_ref as S
from tests.test_step_ops_gpu import Batch, Planned, Trees, _built, accept_reference, check_rotated, i32, raw_of, same  # noqa: F401

pytestmark = pytest.mark.gpu


class Loop:
    """Buffers and calls of a serving loop over n requests with draft trees."""

    def __init__(self, seed, n=5, hq=8, hk=2, d=128, b=16, width=12, blocks=70, nodes=24, rot=None, pairs=False):
        g = self.g = np.random.default_rng(seed)
        self.n, self.hq, self.hk, self.d, self.b, self.width, self.blocks, self.nodes = n, hq, hk, d, b, width, blocks, nodes
        self.freq, self.magnitude = ua.rope_frequencies(rot or d, scaling="linear", factor=2.0)
        self.pairs, self.scale, self.cap = pairs, d ** -0.5, n * nodes
        self.words = -(-nodes // 32)
        self.p = ua.Problem(hq, hk, d, b, blocks, n, width, self.cap, ua.UA_FLAG_CAUSAL, self.scale)
        self.p.set_rope(self.freq, ua.UA_ROPE_PAIRS if pairs else ua.UA_ROPE_HALF, self.magnitude)
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.table, self.held, self.left = z(n, width) - 1, z(n), i32([blocks])
        self.pool = i32(g.permutation(blocks))
        self.ctx, self.new, self.granted, self.cu, self.used = z(n), z(n), z(n), z(n + 1), z(n)
        self.pos, self.slots, self.mask = z(self.cap), z(self.cap, t=torch.int64), z(self.cap, self.words)
        self.parents, self.last, self.path, self.accepted = z(n, nodes), z(n) - 1, z(n, nodes), z(n)
        self.k, self.v = (torch.full((blocks, b, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.qkv = z(self.cap, hq + 2 * hk, d, t=torch.bfloat16)
        self.q_out, self.out = z(self.cap, hq, d, t=torch.bfloat16), z(self.cap, hq, d, t=torch.bfloat16)
        self.ref = S.Step(self.table.tolist(), [0] * n, self.pool.tolist(), b, blocks)
        self.lens = [0] * n
        self.keys = [[] for _ in range(n)]      # per request: (unrotated k row, v row, position) of every kept key

    def draw(self, chain=False):
        g = self.g
        self.trees = [list(range(-1, k - 1)) if chain else S.grow(g, k, 0.6)
                      for k in (int(x) for x in g.integers(0, self.nodes + 1, self.n))]
        self.lasts = [int(g.integers(-1, len(t))) if len(t) else -1 for t in self.trees]
        if chain:
            self.lasts = [len(t) - 1 for t in self.trees]
        rows = torch.zeros(self.n, self.nodes, dtype=torch.int32)
        for s, t in enumerate(self.trees):
            rows[s, :len(t)] = torch.tensor(t, dtype=torch.int32)
        self.parents.copy_(rows)
        self.new.copy_(i32([len(t) for t in self.trees]))
        self.last.copy_(i32(self.lasts))
        self.qkv.copy_(torch.from_numpy(g.normal(size=tuple(self.qkv.shape))).to(torch.bfloat16))

    def calls(self, stream=None):
        hq, hk = self.hq, self.hk
        q, kn, vn = self.qkv.split([hq, hk, hk], 1)
        self.p.plan_step(self.table, self.held, self.pool, self.left, self.ctx, self.new, self.n, self.cap, self.granted,
                         self.cu, self.used, self.pos, self.slots, parents=self.parents, tree_mask=self.mask, stream=stream)
        self.p.rope_store(q, kn, vn, self.pos, self.slots, self.cap, self.k, self.v, q_out=self.q_out, stream=stream)
        most = self.width * self.b
        self.p.forward_tree(self.q_out, self.k, self.v, self.table, self.cu, self.used, self.n, self.cap, self.nodes, most,
                            ua.UA_FLAG_CAUSAL, self.mask, positions=self.pos, out=self.out, stream=stream)
        self.p.cache_accept(self.k, self.v, self.table, self.cu, self.used, self.parents, self.last, self.n, self.cap,
                            self.nodes, most, self.path, self.accepted, self.ctx, stream=stream)

    def state(self):
        return [x.clone() for x in (self.table, self.held, self.left, self.pool, self.ctx, self.k, self.v)]

    def restore(self, state):
        for x, y in zip((self.table, self.held, self.left, self.pool, self.ctx, self.k, self.v), state):
            x.copy_(y)

    def results(self):
        total = int(self.cu[-1])
        return [x.clone() for x in (self.granted, self.cu, self.used, self.pos, self.slots, self.mask[:total], self.path,
                                    self.accepted, self.ctx, self.q_out, self.out[:total], self.k, self.v, self.pool,
                                    self.left, self.held, self.table)]

    def check(self):
        """The last step's results against the references, and the kept keys brought up to date."""
        want, err = self.ref.plan(self.lens, [len(t) for t in self.trees], self.cap, self.trees, self.words)
        assert err == 0 and self.p.check_device_error() == 0
        total = want["cu"][-1]
        same(self.granted, want["granted"])
        same(self.cu, want["cu"])
        same(self.pos, want["pos"] + [0] * (self.cap - total))
        same(self.slots, want["slots"] + [-1] * (self.cap - total))
        x = self.qkv.double().cpu().numpy()
        hq, hk = self.hq, self.hk
        q_rot = self.q_out.double().cpu().numpy()
        check_rotated(q_rot[:total], x[:total, :hq], want["pos"], self.freq, self.pairs, self.magnitude)
        out = self.out.double().cpu().numpy()
        k, v = (t.double().cpu().numpy() for t in (self.k, self.v))
        counts = []
        for s in range(self.n):
            a, z = want["cu"][s], want["cu"][s + 1]
            tree = self.trees[s] if z > a else []
            ctx = self.lens[s]
            new = [(x[t, hq:hq + hk], x[t, hq + hk:], want["pos"][t]) for t in range(a, z)]
            # Attention over the rows as they should lie in the cache: the kept keys and the nodes,
            # rotated, rounded to bf16.
            rows = self.keys[s] + new
            if tree:
                kr = S.rotate(np.stack([r[0] for r in rows]), [r[2] for r in rows], self.freq, self.pairs, self.magnitude)
                vr = np.stack([r[1] for r in rows])
                see = np.array([[c in S.branch(tree, i) for c in range(len(tree))] for i in range(len(tree))])
                o, tot, mag = S.tree_attention(q_rot[a:z], kr, vr, self.scale, see)
                # Keys are bf16 in the cache: 2^-8 of each product.
                dx = R.score_error(mag, self.d) + 2.0 ** -8 * mag
                bound = 2.0 ** -8 * np.abs(o) + (2 * dx + 2.0 ** -10 + 2.0 ** -8) * tot + 1e-30
                assert np.all(np.abs(out[a:z] - o) <= bound), (s, float((np.abs(out[a:z] - o) / bound).max()))
            way = S.branch(tree, self.lasts[s]) if tree else []
            counts.append(len(way))
            self.keys[s] += [new[i] for i in way]
            self.lens[s] = ctx + len(way)
            same(self.path[s, :len(way) + 1][:self.nodes], (way + [-1])[:self.nodes])
            # Every kept key's row is where its position says.
            for j, (kk, vv, at) in enumerate(self.keys[s]):
                assert at == j
                blk, slot = self.ref.table[s][j // self.b], j % self.b
                np.testing.assert_array_equal(v[blk, slot], vv)
                check_rotated(k[blk, slot][None], kk[None], [at], self.freq, self.pairs, self.magnitude)
        same(self.accepted, counts)
        same(self.ctx, self.lens)


@pytest.mark.parametrize("kw", [dict(), dict(blocks=14), dict(hq=4, hk=4, d=64, b=32, width=8, rot=32, pairs=True),
                                dict(hq=16, hk=1, d=256, b=64, width=4, nodes=40, blocks=17)])
def test_a_serving_loop(kw):
    """Prompts as chains, then drafted trees of which a branch is kept, step after step;
    a pool that runs dry on the way, a request that ends and one that takes its place."""
    x = Loop(1, **kw)
    for step in range(7):
        x.draw(chain=step == 0)
        if step == 4:
            x.lens[1], x.keys[1] = 0, []
            x.ctx[1] = 0
        x.calls()
        x.check()
    assert sum(x.lens) > 20


def test_a_captured_step_replayed():
    """One graph of the four calls, replayed on changed inputs, gives what the calls give."""
    x = Loop(2)
    x.draw(chain=True)
    x.calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    before = x.state()
    with torch.cuda.graph(graph):
        x.calls()
    x.restore(before)                                     # (capturing ran nothing)
    for _ in range(3):
        x.draw()
        state = x.state()
        x.calls()
        want = x.results()
        x.restore(state)
        x.out.fill_(5.0)
        graph.replay()
        for a, b in zip(want, x.results()):
            assert torch.equal(a.view(torch.int16) if a.dtype is torch.bfloat16 else a,
                               b.view(torch.int16) if b.dtype is torch.bfloat16 else b)
    assert x.p.check_device_error() == 0


def test_a_step_on_a_side_stream_behind_a_busy_default_stream():
    x = Loop(3)
    x.draw(chain=True)
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    other = torch.ones_like(big)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(60):                                   # about 20 ms of copies
        big.copy_(other)
    x.calls(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    x.check()


def test_two_problems_on_two_streams_at_once():
    """Steps that overlap on the GPU have a problem each."""
    xs = [Loop(4, blocks=90), Loop(5, hq=4, hk=1, blocks=90)]
    streams = [torch.cuda.Stream() for _ in xs]
    for x in xs:
        x.draw(chain=True)
    torch.cuda.synchronize()
    for x, st in zip(xs, streams):
        x.calls(stream=st)
    torch.cuda.synchronize()
    for x in xs:
        x.check()


def test_caches_past_4_gib():
    """Blocks whose bytes and elements lie past 32 bits."""
    hq, hk, d, b, blocks = 16, 8, 256, 64, 40000          # 10.5 GB per cache
    bt = Trees(800, hq, hk, d, b, (9, 20), (150, 90), scale=None)
    far = np.arange(blocks - bt.blocks, blocks)
    kc, vc = (torch.zeros(blocks, b, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt.device()
    kc[far], vc[far] = bt.d_k, bt.d_v
    bt.d_table = torch.where(bt.d_table >= 0, bt.d_table + int(far[0]), bt.d_table)
    p = ua.Problem(hq, hk, d, b, blocks, 2, bt.width, 64, ua.UA_FLAG_CAUSAL, bt.scale)
    bt.d_k, bt.d_v = kc, vc
    bt.check(bt.run(p, ua.UA_FLAG_CAUSAL, pos=False))
    assert p.check_device_error() == 0
    # The accepted branches, then new keys at far slots.
    trees = bt.trees
    last = [8, 19]
    path, acc, used = torch.zeros(2, 20, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([0, 0])
    parents = i32([t + [-1] * (20 - len(t)) for t in trees])
    p.cache_accept(kc, vc, bt.d_table, bt.d_cu, bt.d_sk, parents, i32(last), 2, 29, 20, 150, path, acc, used)
    want, count = accept_reference(bt, trees, last, 20)
    same(path, want)
    np.testing.assert_array_equal(raw_of(kc[far], "bf16"), bt.kc.raw)
    np.testing.assert_array_equal(raw_of(vc[far], "bf16"), bt.vc.raw)
    p.set_rope([1.0] * 8)
    rows = torch.randn(3, hq + 2 * hk, d, device="cuda").to(torch.bfloat16)
    q, kn, vn = rows.split([hq, hk, hk], 1)
    slots = torch.tensor([blocks * b - 1, (blocks - 2) * b + 5, 3], device="cuda")
    p.rope_store(q, kn, vn, i32([0, 0, 0]), slots, 3, kc, vc)
    assert p.check_device_error() == 0
    assert torch.equal(kc.view(-1, hk, d)[slots], kn) and torch.equal(vc.view(-1, hk, d)[slots], vn)


@pytest.mark.parametrize("hq,hk,d,sq,sk", [(4, 1, 64, 5, 30000), (16, 1, 128, 40, 9000), (2, 1, 256, 3, 12000)])
def test_long_requests_are_cut_into_many_pieces(hq, hk, d, sq, sk):
    bt = Trees(810 + d, hq, hk, d, 64, (sq,), (sk,)).device()
    p = bt.problem()
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == 0
    bt.check(got)
    for _ in range(3):                                    # one order of addition
        assert torch.equal(bt.run(p, ua.UA_FLAG_CAUSAL, pos=False), got)


def test_uneven_batches():
    """One long request among short ones, and requests without nodes."""
    sk = [20, 6000, 3, 1, 64, 65, 130, 9, 700, 2]
    sq = [5, 33, 3, 1, 64, 1, 0, 9, 40, 2]
    for hq, hk, d in ((8, 2, 128), (8, 4, 64), (4, 2, 256)):
        bt = Trees(820 + d, hq, hk, d, 16, sq, sk).device()
        p = bt.problem(split_partials=ua.UA_PARTIALS_BF16 if d == 64 else ua.UA_PARTIALS_F32)
        got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
        assert p.check_device_error() == 0
        bt.check(got, bf16_parts=d == 64)


def test_a_problem_for_key_weights_has_fewer_shares():
    bt = Trees(830, 8, 2, 64, 16, (3, 4), (900, 2000)).device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == 0
    bt.check(got)


@pytest.mark.parametrize("weights", [0, ua.UA_FLAG_KEY_WEIGHTS])
@pytest.mark.parametrize("hq,hk,d,sq,sk", [(1, 1, 64, 1, 3000), (2, 1, 256, 3, 777), (4, 4, 128, 2, 1500)])
def test_bounds_far_above_the_call(hq, hk, d, sq, sk, weights):
    """max_seqlen_q of 64 nodes where the problem has room for a few tokens: partials are
    as long as the tokens are many."""
    bt = Trees(832, hq, hk, d, 16, (sq,), (sk,), words=2).device()
    width = bt.d_table.shape[1]
    p = ua.Problem(hq, hk, d, 16, bt.d_k.shape[0], 1, width, sq, ua.UA_FLAG_CAUSAL | weights, bt.scale)
    got = p.forward_tree(bt.d_q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 1, sq, 64, width * 16, ua.UA_FLAG_CAUSAL,
                         torch.from_numpy(bt.mask.view(np.int32)).cuda())
    assert p.check_device_error() == 0
    bt.check(got)


def test_each_call_sees_what_the_one_in_front_wrote():
    """Kernels start under the end of the one in front, which has had the same lines
    of the tables, lengths and masks in its hands."""
    loop = Loop(833, n=24, width=16, blocks=400, nodes=16)
    busy = torch.randn(1 << 22, device="cuda")
    for _ in range(6):
        loop.draw()
        before = [x.clone() for x in (loop.table, loop.held, loop.pool, loop.left, loop.ctx, loop.k, loop.v)]
        loop.calls()
        fast = [x.clone() for x in (loop.table, loop.pos, loop.slots, loop.mask, loop.out, loop.path, loop.ctx, loop.k, loop.v)]
        for x, y in zip((loop.table, loop.held, loop.pool, loop.left, loop.ctx, loop.k, loop.v), before):
            x.copy_(y)
        # The same calls, each behind a complete stop.
        real = {name: getattr(loop.p, name) for name in ("plan_step", "rope_store", "forward_tree", "cache_accept")}
        for name, call in real.items():
            def slow(*a, call=call, **kw):
                busy.sin_()
                torch.cuda.synchronize()
                out = call(*a, **kw)
                torch.cuda.synchronize()
                return out
            setattr(loop.p, name, slow)
        loop.calls()
        for name in real:
            delattr(loop.p, name)
        for x, y in zip((loop.table, loop.pos, loop.slots, loop.mask, loop.out, loop.path, loop.ctx, loop.k, loop.v), fast):
            torch.testing.assert_close(x, y, rtol=0, atol=0, equal_nan=True)
    assert loop.p.check_device_error() == 0


def test_calls_without_anything_to_do():
    bt = Trees(831, 8, 2, 128, 16, (2, 3), (40, 20)).device()
    p = bt.problem()
    out = torch.full_like(bt.d_q, 7.0)
    args = bt.d_q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    for n, total in ((0, 5), (2, 0)):
        p.forward_tree(*args, n, total, 3, 40, ua.UA_FLAG_CAUSAL, mask, out=out)
        assert p.last_launch_count() == 0
    # No rows allowed: every sequence is too long.
    p.forward_tree(*args, 2, 5, 0, 40, ua.UA_FLAG_CAUSAL, mask, out=out)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS or bool((out == 7).all())


@pytest.mark.parametrize("seed", range(24))
def test_random_trees(seed):
    g = np.random.default_rng(6000 + seed)
    hk = int(g.choice([1, 2, 3, 8]))
    gq = int(g.choice([1, 2, 3, 4, 8, 16]))
    d, b = int(g.choice([64, 128, 256])), int(g.choice([16, 32, 64]))
    n = int(g.integers(1, 7))
    sq = [int(x) for x in np.minimum(np.exp(g.uniform(0, 5, n)), 70 if gq < 8 else 40)]
    sk = [a + int(np.exp(g.uniform(0, 7))) - 1 for a in sq]
    softcap = float(g.choice([0.0, 0.0, 8.0]))
    window = int(g.choice([0, 0, 1, 5, 60, 500]))
    sinks = g.normal(size=gq * hk).astype(np.float32) if g.random() < 0.4 else None
    alibi = (2.0 ** -g.uniform(0, 8, gq * hk)).astype(np.float32) if g.random() < 0.3 else None
    bt = Trees(7000 + seed, gq * hk, hk, d, b, sq, sk)
    if g.random() < 0.3:
        bt.mask = bt.rng.integers(0, 1 << 32, bt.mask.shape, dtype=np.uint64).astype(np.uint32)
    bt.device()
    flags = ua.flags_of(True, softcap, alibi is not None, window, sinks is not None)
    p = bt.problem(flags, softcap=softcap, window=window)
    got = bt.run(p, flags, sinks, alibi)
    assert p.check_device_error() == 0
    bt.check(got, softcap, window=window, sinks=sinks, alibi=alibi)


@pytest.mark.parametrize("seed", range(12))
def test_random_plans(seed):
    g = np.random.default_rng(8000 + seed)
    n, b = int(g.integers(1, 400)), int(g.choice([16, 32, 64]))
    ctx = [int(x) for x in g.integers(0, 12 * b, n)]
    st = Planned(8100 + seed, n, b, width=16, num_blocks=13 * n + 500, pool=int(g.integers(0, 400)), ctx=ctx,
                 spare=int(g.integers(0, 3)))
    tree = g.random() < 0.5
    for _ in range(3):
        most = min(70, 2 * b)
        new = [min(int(x), 16 * b - c) for x, c in zip(g.integers(0, most, n), st.ctx)]
        trees = [S.grow(g, k) for k in new] if tree else None
        out, want = st.step(new, sum(new) + int(g.integers(0, 9)), trees, 3 if tree else 0)
        st.ctx = [max(0, u - int(g.integers(0, 3 * b))) for u in want["used"]]
