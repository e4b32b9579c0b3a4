"""Rotary stores over random shapes, strides, positions and slots, against the 64-bit rotation of
tests/step_ref.py and the stored bytes of tests/cache_ref.py.  Tolerances:
tests/test_step_ops_gpu.py."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests import step_ref as S
from tests.test_step_ops_gpu import _built, bits, check_rotated, i32, raw_of, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = dict(bf16=ua.UA_DTYPE_BF16, fp8=ua.UA_DTYPE_FP8_E4M3, fp4=ua.UA_DTYPE_FP4_E2M1)


def rows_of(x, fused):
    """q, k and v of a token behind each other, or tensors of their own with room between tokens."""
    if fused is not None:
        return torch.cat(x, 1).split(fused, 1)
    out = []
    for i, t in enumerate(x):
        n, h, d = t.shape
        wide = torch.full((n, h * d + (8 if i else 24)), 9.0, dtype=t.dtype, device=t.device)
        wide[:, :h * d] = t.flatten(1)
        out.append(wide.as_strided((n, h, d), (wide.stride(0), d, 1)))
    return out


@pytest.mark.parametrize("seed", range(48))
def test_random_rotary_stores(seed):
    g = np.random.default_rng(3000 + seed)
    kv = ["bf16", "fp8", "fp4"][seed % 3]
    d = 128 if kv == "fp8" else int(g.choice([64, 128, 256]))
    hk = int(np.exp(g.uniform(0, np.log(12))))
    hq = hk * int(g.choice([1, 2, 3, 4, 8]))
    b, n = int(g.choice([16, 32, 64])), int(np.exp(g.uniform(0, np.log(300 if kv == "bf16" else 120))))
    rot, pairs, in_place = 16 * int(g.integers(1, d // 16 + 1)), bool(g.random() < 0.5), bool(g.random() < 0.4)
    scaling = [{}, dict(scaling="linear", factor=3.0), dict(scaling="bands", factor=8.0, trained=8192),
               dict(scaling="yarn", factor=16.0, trained=4096, high=32.0)][int(g.integers(4))]
    freq, magnitude = ua.rope_frequencies(rot, base=float(g.choice([10000.0, 500000.0])), **scaling)
    kscale, vscale = (float(x) for x in (g.choice([0.25, 1.0, 0.03, 1.7], 2) if kv != "bf16" else (1.0, 1.0)))
    blocks = n // b + 2
    pos = np.where(g.random(n) < 0.5, g.integers(0, 200000, n), g.integers(-2 ** 31, 2 ** 31, n))
    slots = g.permutation(blocks * b)[:n]
    slots[g.random(n) < 0.15] = -1
    past = bool(g.random() < 0.3)
    if past:
        slots[0] = blocks * b + int(g.integers(0, 1 << 40))
    _, x = bits(g.normal(size=(n, hq + 2 * hk, d)) * np.exp(g.uniform(-3, 3, (n, 1, 1))))
    dev = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()
    q, kn, vn = rows_of(dev.split([hq, hk, hk], 1), [hq, hk, hk] if g.random() < 0.5 else None)
    behind = [(t, t.untyped_storage(), t.untyped_storage().nbytes()) for t in (q, kn, vn)]
    before = [torch.tensor([], dtype=torch.bfloat16, device="cuda").set_(s).clone() for _, s, _ in behind]
    p = ua.Problem(hq, hk, d, b, blocks, 1, 8, n, ua.UA_FLAG_CAUSAL, 0.1, kv_dtype=TYPES[kv], k_scale=kscale, v_scale=vscale)
    p.set_rope(freq, int(pairs), magnitude)
    kc, vc = (R.Cache(kv, blocks, b, hk, d, s, 0x55) for s in (kscale, vscale))
    d_k, d_v = to_gpu(kc), to_gpu(vc)
    d_slots = torch.from_numpy(slots).cuda()
    # The rotated keys as bf16, in the order of the tokens.
    p16 = ua.Problem(hq, hk, d, 16, n // 16 + 1, 1, 8, n, ua.UA_FLAG_CAUSAL, 0.1)
    p16.set_rope(freq, int(pairs), magnitude)
    k16 = torch.zeros(n // 16 + 1, 16, hk, d, dtype=torch.bfloat16, device="cuda")
    p16.rope_store(q, kn, vn, i32(pos), torch.arange(n, device="cuda"), n, k16, torch.zeros_like(k16))
    k_rot = k16.view(-1, hk, d)[:n]
    check_rotated(k_rot.double().cpu().numpy(), x[:, hq:hq + hk], pos, freq, pairs, magnitude)

    out = p.rope_store(q, kn, vn, i32(pos), d_slots, n, d_k, d_v, q_out=q if in_place else None)
    assert p.check_device_error() == (S.BLOCK_ID if past else 0)
    check_rotated(out.double().cpu().numpy(), x[:, :hq], pos, freq, pairs, magnitude)
    # Nothing else of the inputs changed: with q turned back, all of their memory is as it was.
    if in_place:
        q.copy_(dev[:, :hq])
    for (_, s, _), old in zip(behind, before):
        assert torch.equal(torch.tensor([], dtype=torch.bfloat16, device="cuda").set_(s).view(torch.int16), old.view(torch.int16))
    kb, vb = (t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16) for t in (k_rot, vn))
    kr, vr = R.bf16_values(k_rot), R.bf16_values(vn)
    for t in range(n):
        if 0 <= slots[t] < blocks * b:
            at = divmod(int(slots[t]), b)
            kc.put(*at, kr[t], kb[t])
            vc.put(*at, vr[t], vb[t])
    np.testing.assert_array_equal(raw_of(d_k, kv), kc.raw)
    np.testing.assert_array_equal(raw_of(d_v, kv), vc.raw)
