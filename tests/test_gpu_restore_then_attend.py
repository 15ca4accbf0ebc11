"""A restore of several launches with serving calls right behind it on the
stream: a cache that is kept as containers is restored, written to and
attended in one go.  The calls are ordered behind all of the restore's
launches, not its last one alone, so the results have the bits that they have
with a synchronization in between.
"""
import math

import numpy as np
import pytest

from weight_streaming_canonical_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [40, 1024])
def test_a_restored_cache_is_written_and_attended_at_once(afx, pages):
    import torch
    page, heads, dim, tokens = 64, 2, 128, 3
    n = pages * page * heads * dim
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    # two large BF16 containers (one launch), then small FP16 and E4M3 ones (one launch each, the last to start)
    coded = [afx.encode(synth.normal(n, seed=i)) for i in (1, 2)]
    coded += [afx.encode(synth.normal_fp16(5000, seed=3), fmt=afx.AFX_FMT_FP16),
              afx.encode(synth.normal_e4m3(5000, seed=4), fmt=afx.AFX_FMT_E4M3)]
    containers, descs = [cuda(c) for c, _ in coded], [d for _, d in coded]
    pools = [torch.empty((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [p.view(torch.int16).view(-1) for p in pools] + [torch.empty(5000, dtype=torch.int16, device="cuda"),
                                                            torch.empty(5000, dtype=torch.uint8, device="cuda")]
    cache = afx.kv_cache(*pools)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = (torch.randn((tokens, 10, dim), device="cuda")).to(torch.bfloat16)
    k, v = [torch.randn((tokens, heads, dim), device="cuda").to(torch.bfloat16) for _ in range(2)]
    # the new tokens are the last of the last page, behind which the restore's last CTAs lie
    length = pages * page
    slots, starts, lens, table = ints([length - tokens + i for i in range(tokens)]), ints([0, tokens]), ints([length]), ints([list(range(pages))])
    args = afx.attention_args(cache, 10, tokens, starts, lens, table, 1 / math.sqrt(dim))
    ws = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    afx.afx_attention_plan(args, ws)

    def run(wait):
        out, lse = torch.empty_like(q), torch.empty((tokens, 10), device="cuda")
        for p in pools:
            p.fill_(math.nan)
        afx.afx_decode_batch(descs, containers, outs, status_dev=status)
        if wait:
            torch.cuda.synchronize()
        afx.afx_kv_write(cache, k, v, slots, status_dev=status)
        afx.afx_attention(args, q, out, ws, lse=lse, status_dev=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        return out, lse, [p.clone() for p in pools]

    want = run(True)
    assert torch.isfinite(want[0]).all() and torch.equal(want[2][0][-1, -tokens:], k)
    for _ in range(20):
        out, lse, after = run(False)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(after[0].view(torch.int16), want[2][0].view(torch.int16))
        assert torch.equal(after[1].view(torch.int16), want[2][1].view(torch.int16))
