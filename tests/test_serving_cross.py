"""Cross attention within a serving loop, at its own tolerances: rows that were written, forked and
compacted, read by runs of queries.  test_serving_run.py allows every attention call what the
decode kernels need; here test_cross.py's counts of roundings stand alone, and the errors' 2-norm
stays below 2^-8 of the result's."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_07_b200 import tqkv
from test_serving_run import Loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("runs", [[3, 20, 0, 1, 40, 2], [2, 4, 0, 1, 3, 2]])
@pytest.mark.parametrize("d,kbits,P,H,G", [(64, 4, 16, 2, 2), (128, 2, 64, 2, 4), (128, 8, 64, 1, 2)])
def test_runs_over_forked_and_compacted_rows(d, kbits, P, H, G, runs):
    s = Loop(d, kbits, P, H, G, seed=3)
    prompt = [90, 70, 0, 0, 0, 0]
    slots = s.ints([-7] * sum(prompt))
    s.reserve(s.ints(prompt), slots)
    pos = s.ints(list(range(90)) + list(range(70)))
    for c in s.caches:
        q, k, v = s.project(sum(prompt))
        _, kn = tqkv.qk_norm_rope(s.rope, q, k, pos, s.inv, *s.w)
        tqkv.encode(s.cd.kp, s.cd.vp, s.cd.desc, kn, v, slots, c)
    tqkv.pages_fork(s.cd.desc, s.caches, s.refs, s.table, s.lens, s.ints([0, 1, 1]), s.ints([2, 3, 4]), workspace=s.ws)
    keep = torch.zeros((2, 60), dtype=torch.int32, device=s.lens.device)
    keep[0, :50], keep[1] = torch.arange(40, 90), torch.arange(59, -1, -1)
    tqkv.pages_compact(s.cd.desc, s.caches, s.refs, s.table, s.lens, s.ints([2, 4]), keep, s.ints([50, 60]), workspace=s.ws)
    assert s.lens.tolist() == [90, 70, 50, 70, 60, 0] and tqkv.read_status(s.ws) == 0
    cu, most = s.ints([0] + list(np.cumsum(runs))), max(runs)
    for c in s.caches:
        q, _, _ = s.project(sum(runs))
        q = q.contiguous()
        out = tqkv.cross_attn(s.cd.kp, s.cd.vp, s.cd.desc, q, cu, most, s.table, s.lens, s.width * s.P, c)
        raw, Q, got = c.view(-1, c.shape[-1]).cpu().numpy(), q.double().cpu().numpy(), out.double().cpu().numpy()
        err2 = ref2 = 0.0
        for i, r in enumerate(r for r, m in enumerate(runs) for _ in range(m)):
            for h in range(H):
                hs = slice(h * G, (h + 1) * G)
                ref, _, tol, _ = s.cd.attend(Q[i, hs], *s.cd.states(raw, s.slots_of(r), h))
                e = np.abs(got[i, hs] - ref)
                assert (e <= tol).all(), (r, (e / np.maximum(tol, 1e-300)).max())
                err2, ref2 = err2 + (e ** 2).sum(), ref2 + (ref ** 2).sum()
        assert err2 <= 2.0 ** -16 * ref2, math.sqrt(err2 / ref2)
