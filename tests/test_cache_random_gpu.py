"""Seeded random calls of the cache operators over their whole ranges: head layouts, head
and block sizes, lengths from zero, masks and score terms, strides, budgets, against the
64-bit implementations.  Tolerances: tests/test_cache_ops_gpu.py."""
import random

import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests.test_cache_long_gpu import LongBatch, check, check_weights
from tests.test_cache_ops_gpu import Batch, DT, _built, evict_weights, raw_of, terms  # noqa: F401

pytestmark = pytest.mark.gpu


def log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def attention_call(rng, kind):
    d = 128 if kind == "fp8" else rng.choice([64, 128, 256])
    g = rng.choice([1, 2, 3, 4, 5, 8, 16] + ([12, 24, 40, 130] if kind == "fp4" else []))
    hk = rng.choice([1, 2, 3, 8]) if g < 100 else 1
    n = log_int(rng, 1, 24)
    top = log_int(rng, 2, 6000 if g < 24 else 800)
    most = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 90)])
    sq = [rng.choice([0, rng.randint(1, most), rng.randint(1, most), most]) for _ in range(n)]
    sk = [q + rng.choice([0, rng.randint(0, top)]) for q in sq]
    if not sum(sq):
        sq[0] = sk[0] = 1
    causal = rng.random() < 0.9
    kw = dict(causal=causal, softcap=rng.choice([0.0, 0.0, 25.0]), alibi=rng.random() < 0.25,
              window=rng.choice([0, 0, log_int(rng, 1, 2000)]) if causal else 0, sinks=rng.random() < 0.3)
    return g * hk, hk, d, rng.choice([16, 32, 64]), sq, sk, kw


@pytest.mark.parametrize("kind", ["fp4", "bf16", "fp8"])
@pytest.mark.parametrize("part", range(4))
def test_random_attention_with_key_weights(kind, part):
    for call in range(24 if kind == "fp4" else 12):
        rng = random.Random("%s %d %d" % (kind, part, call))
        hq, hk, d, b, sq, sk, kw = attention_call(rng, kind)
        bt = LongBatch(rng.randrange(1 << 30), kind, hq, hk, d, b, sq, sk, qmax=rng.choice([0.01, 1.0, 3.0]))
        flags, softcap, window, sinks, alibi = terms(hq, **kw)
        dev = [None if x is None else torch.from_numpy(x).cuda() for x in (sinks, alibi)]
        bf16_parts = rng.random() < 0.2
        p = bt.problem(flags | ua.UA_FLAG_KEY_WEIGHTS, softcap=softcap, window=window,
                       split_partials=ua.UA_PARTIALS_BF16 if bf16_parts else ua.UA_PARTIALS_F32)
        n, most, decay = bt.n, max(max(sk), 1), rng.choice([0.0, 0.7, 1.0])
        w_in = torch.empty(n, hk, most + rng.randint(0, 9), device="cuda").exponential_(generator=bt.gen)
        w = torch.full_like(w_in, -7.0)
        what = (kind, part, call, hq, hk, d, b, sq, sk, kw)
        outs = [p.forward_weights(*bt.args(), flags, w_in, w, decay=decay, sinks=dev[0], alibi_slopes=dev[1])]
        if kind == "fp4":
            outs.append(p.forward(*bt.args(), flags, *dev))
        assert p.check_device_error() == 0, what
        extra = most if alibi is not None else 0.0
        for s in range(n):
            k = sk[s]
            if not sq[s]:
                assert bool((w[s] == -7.0).all()), what
                continue
            ref = bt.reference(s, kw["causal"], softcap, window, sinks, alibi)
            old = torch.where(torch.arange(k, device="cuda") < k - sq[s], decay * w_in[s, :, :k].double(), 0.0)
            check_weights(bt, s, w[s, :, :k], old, ref, softcap, extra)
            assert bool((w[s, :, k:] == -7.0).all()), what
            for out in outs:
                check(bt, s, out, ref, softcap, extra, bf16_p=kind == "bf16" or bf16_parts)


@pytest.mark.parametrize("part", range(4))
def test_random_evictions(part):
    for call in range(16):
        rng = random.Random("evict %d %d" % (part, call))
        kind = rng.choice(["fp4", "bf16", "fp8"])
        d, b, hk = rng.choice([64, 128, 256]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3])
        n = log_int(rng, 1, 12)
        top = log_int(rng, 2, 3000)
        sk = [rng.choice([0, top, rng.randint(0, top)]) for _ in range(n)]
        budget = log_int(rng, 1, 2 * top)
        recent = rng.choice([0, budget, rng.randint(0, budget)])
        g = torch.Generator(device="cuda").manual_seed(rng.randrange(1 << 30))
        nblk = [-(-k // b) for k in sk]
        kblk = [-(-min(k, budget) // b) for k in sk]
        blocks, width = sum(nblk) + sum(kblk) + 1, max(max(nblk), 1) + 1
        ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        to = table.clone()
        off = 0
        for s in range(n):
            table[s, :nblk[s]] = ids[off:off + nblk[s]]
            to[s, :kblk[s]] = ids[off + nblk[s]:off + nblk[s] + kblk[s]]
            off += nblk[s] + kblk[s]
        in_place, same_w = rng.random() < 0.5, rng.random() < 0.5
        to = table if in_place else to
        shape = ua.cache_shape(blocks, hk, d, b, DT[kind])
        k, v = (torch.randint(0, 1 << 15, shape, generator=g, device="cuda").to(torch.int16 if kind == "bf16"
                                                                                 else torch.uint8) for _ in range(2))
        k0, v0 = k.clone(), v.clone()
        w = evict_weights(np.random.default_rng(rng.randrange(1 << 30)), (n, hk, max(max(sk), 4) + rng.randint(0, 9)))
        dw = torch.from_numpy(w).cuda()
        dwo = dw if same_w else torch.full_like(dw, 5.0)
        kept = torch.full((n, hk, budget), 99, dtype=torch.int32, device="cuda")
        used = torch.tensor(sk, dtype=torch.int32, device="cuda")
        used_out = used if rng.random() < 0.5 else torch.full_like(used, 77)
        p = ua.Problem(hk, hk, d, b, blocks, n, width, 1, ua.UA_FLAG_CAUSAL, 0.1, kv_dtype=DT["bf16" if kind == "fp8"
                       and d != 128 else kind])
        if kind == "fp8" and d != 128:
            continue                                   # an fp8 cache has d = 128
        p.cache_evict(k, v, table, used, n, max(sk), dw, dwo, budget, recent, kept, used_out,
                      dst_block_table=None if in_place else to)
        assert p.check_device_error() == 0
        assert used_out.tolist() == [min(x, budget) for x in sk]
        for s in range(n):
            for h in range(hk):
                want = R.evict_choice(w[s, h], sk[s], budget, recent)
                m = len(want)
                np.testing.assert_array_equal(kept[s, h].cpu().numpy(), np.append(want, [-1] * (budget - m)))
                np.testing.assert_array_equal(dwo[s, h, :m].cpu().numpy(), w[s, h][want])
                at = torch.from_numpy(want).cuda()
                r = torch.arange(m, device="cuda")
                for now, old in ((k, k0), (v, v0)):
                    if kind == "fp4":
                        c, e = b * d // 2, torch.arange(d // 2, device="cuda")
                        for base, size in ((0, d // 2), (c, d // 16)):
                            x = now[to[s, r // b].long()[:, None], h, base + (r % b)[:, None] * size + e[:size]]
                            y = old[table[s, at // b].long()[:, None], h, base + (at % b)[:, None] * size + e[:size]]
                            assert torch.equal(x, y)
                    else:
                        assert torch.equal(now[to[s, r // b].long(), r % b, h],
                                           old[table[s, at // b].long(), at % b, h])


@pytest.mark.parametrize("part", range(3))
def test_random_stores_and_expansions(part):
    for call in range(8):
        rng = random.Random("store %d %d" % (part, call))
        kind = rng.choice(["fp4", "fp4", "fp8", "bf16"])
        d = 128 if kind == "fp8" else rng.choice([64, 128, 256])
        b, hk, n = rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 5]), rng.randint(1, 5)
        sq = [rng.choice([0, 1, rng.randint(1, 70)]) for _ in range(n)]
        sk = [q + rng.choice([0, rng.randint(0, 90)]) for q in sq]
        if not sum(sq):
            sq[0], sk[0] = 1, sk[0] + 1
        ks, vs = (rng.choice([1.0, 0.5, 2.0 ** -20, 0.05, 3.0, 1e-3, 700.0]) for _ in range(2))
        bt = Batch(rng.randrange(1 << 30), kind, 2 * hk, hk, d, b, sq, sk, ks, vs, store=False,
                   std=rng.choice([1.0, 1e-3, 200.0])).device()
        for s in range(n):
            for j in range(sk[s] - sq[s], sk[s]):
                bt.put(s, j)
        p = bt.problem(max_total_q=sum(sq) + 3)
        pad = rng.choice([0, 8, 24]) if hk > 1 else 0
        fused = torch.zeros(sum(sq) + 2, hk * d + pad, dtype=torch.bfloat16, device="cuda")
        kn = fused[:, :hk * d].unflatten(1, (hk, d))
        vn = torch.zeros_like(fused)[:, :hk * d].unflatten(1, (hk, d))
        kn[:sum(sq)], vn[:sum(sq)] = bt.new_rows("k"), bt.new_rows("v")
        p.cache_store(kn, vn, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, n, sum(sq), max(sq), max(sk))
        assert p.check_device_error() == 0
        np.testing.assert_array_equal(raw_of(bt.d_k, kind), bt.kc.raw)
        np.testing.assert_array_equal(raw_of(bt.d_v, kind), bt.vc.raw)
        # And back: the new keys alone, into other pages.
        width = bt.width + rng.randint(0, 3)
        pages = [torch.full((bt.blocks + 1, b, hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        table = np.full((n, width), -1, np.int32)
        table[:, :bt.width] = bt.table
        table = torch.from_numpy(np.where(table >= 0, bt.blocks - table, -1).astype(np.int32)).cuda()
        begin = torch.tensor([k - q for q, k in zip(sq, sk)], dtype=torch.int32, device="cuda")
        p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, n, max(sq), *pages, table, begin=begin)
        assert p.check_device_error() == 0
        for c, page in ((bt.kc, pages[0]), (bt.vc, pages[1])):
            got = page.double().cpu().numpy()
            want, seen = np.full(got.shape, 7.0), np.zeros(got.shape[:2], bool)
            for s in range(n):
                for j in range(sk[s] - sq[s], sk[s]):
                    at = bt.blocks - int(bt.table[s, j // b]), j % b
                    want[at], seen[at] = c.row(int(bt.table[s, j // b]), j % b), True
            assert np.all(got[~seen] == 7.0)
            # The fp32 product (half a step: 2^-24), rounded to bf16 (2^-8).
            assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 1e-40)
