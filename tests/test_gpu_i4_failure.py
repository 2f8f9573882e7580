"""The bounded waits of the tcgen05 prefix pass over a 4-bit pool, without a
fault: with a limit of 1 ns (padoc_debug_set_wait_limit) its waits run out, every
role leaves its loop, the decoders wait for their copies and the issuers for
their products, tensor memory is freed and the kernel ends.  padoc_device_status
reports PADOC_ERR_DEVICE_TIMEOUT, and with the default limit the same steps
match the float64 oracle again."""
import pytest

from oracle import tree_attention as ta
from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

from test_gpu_i4_decode import cached, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [5, 6])
def test_prefix_pass_wait_timeout_is_reported_and_recovered(padoc_lib, seed):
    import torch
    from tree_structured_shared_gb300 import harness
    # several units a CTA, of one to six tiles
    pages = [wl.DecodePage(P, [P] * 4, [9, 0, 30, 2], [5, 3, 8, 4], [[-1] + list(range(n - 1)) for n in (5, 3, 8, 4)])
             for P in [700, 100, 130, 300] * 12]
    w = wl.DecodeWorkload("t", pages, 8, 2, 128, 0.7)
    vals = wl.decode_values(w, seed)
    d = harness.Decode(w, vals, dtype=padoc.I4)
    padoc.device_status()
    padoc.debug_set_wait_limit(1)
    try:
        d.run()
        torch.cuda.synchronize()
        with pytest.raises(padoc.PadocError) as e:
            padoc.device_status()
        assert e.value.code == padoc.ERR_DEVICE_TIMEOUT
    finally:
        padoc.debug_set_wait_limit(0)
    padoc.device_status()
    c = cached(vals)
    O, L = ta.branch_decode(w, c)
    for _ in range(2):
        o, lse = d.run()
        torch.cuda.synchronize()
        padoc.device_status()
        check(o.float().cpu().numpy()[: w.n_queries], lse.cpu().numpy()[: w.n_queries], O, L, c, what="after a timeout")
