"""What a call that gave up in a wait leaves for the next replay of its graph.  A captured call counts its split
units' arrivals under the same tag in every replay, so a replay that is reported as timed out must not leave a
count behind: the next one would take it up, merge partials of the one before and report nothing."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref, check_attention

pytestmark = pytest.mark.gpu

LIMITS = [1, 200, 500, 800, 1200, 1600, 2000, 2500, 3000, 4000, 6000]   # cycles; the first waits take 500 to 4000


def counts(ws, units):
    """The arrivals of each unit, the lower 16 bits of its counter; the counters are first in the workspace."""
    return (ws[:units * 8].view(torch.int64) & 0xFFFF).tolist()


class Call:
    def __init__(self, paged, B, Hq, Hkv, Sq, S, D, P=64):
        g = torch.Generator().manual_seed(S)
        self.q, self.k, self.v = (torch.randn(*s, generator=g).to(torch.bfloat16) for s in ((B, Hq, Sq, D), (B, Hkv, S, D), (B, Hkv, S, D)))
        q, k, v = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.lens, self.scale = [S] * B, D ** -0.5
        self.out, self.lse = torch.empty_like(q), torch.empty(B, Hq, Sq, device="cuda")
        if paged:
            width = S // P
            pools = [x.view(B, Hkv, width, P, D).transpose(1, 2).reshape(B * width, Hkv, P, D) for x in (k, v)]
            cache = F.make_kv_cache(*pools)
            table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
            lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
            self.units = B * Hkv * -(-Hq // Hkv * Sq // 16)
            n = F.fmha_paged_workspace_size(B, Hq, Sq, cache, F.make_opts())
            self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
            opts = F.make_opts(workspace=self.ws)
            self.call = lambda: F.fmha_fwd_paged(q, cache, table, lens, self.out, self.lse, self.scale, opts)
        else:
            self.units = B * Hkv
            self.ws = torch.zeros(F.fmha_workspace_size(B, Hq, Hkv, Sq, S, D, F.make_opts()), dtype=torch.uint8, device="cuda")
            opts = F.make_opts(workspace=self.ws)
            self.call = lambda: F.fmha_fwd_ex(q, k, v, self.out, self.lse, self.scale, opts)
        self.ref = attention_ref(self.q, self.k, self.v, self.lens, self.scale, False)

    def right(self, paged, what):
        if paged:
            check_attention(self.out, self.lse, self.ref, what=what)
        else:   # weights rounded once to BF16: half a step, 2^-8 of sum_j p_j |v_j|, on top
            o, _, a = self.ref
            d = (self.out.double().cpu() - o).abs()
            assert (d <= a * (2.0 ** -8 + 2.0 ** -11) + 2.0 ** -8 * o.abs()).all(), f"{what}: off by {d.max():.3e}"


@pytest.mark.parametrize("paged, B, Hq, Hkv, Sq, S, D", [
    (False, 2, 8, 8, 1, 2048, 128),    # one column, the softmax warps' own epilogue
    (False, 1, 16, 1, 1, 5120, 64),    # sixteen columns, epilogue warps
    (True, 2, 8, 8, 1, 2048, 128), (True, 1, 16, 1, 1, 5120, 64), (True, 1, 32, 8, 1, 4096, 128)])
def test_no_arrivals_left_by_a_call_that_timed_out(paged, B, Hq, Hkv, Sq, S, D):
    c = Call(paged, B, Hq, Hkv, Sq, S, D)
    c.call()
    assert F.fmha_check_status() == 0 and counts(c.ws, c.units) == [0] * c.units
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    late, stream = 0, torch.cuda.Stream()
    for limit in LIMITS:
        with torch.cuda.stream(stream):
            F.fmha_set_wait_limit(limit)
            try:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    c.call()
            finally:
                F.fmha_set_wait_limit(0)
            for turn in range(6):
                if turn % 2 == 0:
                    flush.fill_(turn)     # the keys leave L2: longer waits
                c.out.fill_(float("nan"))
                c.lse.fill_(float("nan"))
                g.replay()
                rc = F.fmha_check_status(stream)
                assert rc in (F.FMHA_OK, F.FMHA_ERR_TIMEOUT)
                late += rc == F.FMHA_ERR_TIMEOUT
                left = counts(c.ws, c.units)
                assert left == [0] * c.units, f"limit {limit}, turn {turn}, status {rc}: {left}"
                if rc == F.FMHA_OK:
                    c.right(paged, f"limit {limit}, turn {turn}")
    assert late > 0
    with torch.cuda.stream(stream):
        c.call()
        assert F.fmha_check_status(stream) == 0
    c.right(paged, "afterwards")
