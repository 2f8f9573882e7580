"""The bounded waits of the loss kernel, without a fault: with a limit of 1 ns
(padoc_debug_set_wait_limit) its waits run out, every role of both CTAs of a pair leaves
its loop, the issuer waits for its products and the CTAs for their copies, tensor memory
is freed and the kernel ends.  padoc_device_status reports PADOC_ERR_DEVICE_TIMEOUT, and
with the default limit the same calls match the definition again."""
import pytest

from tree_structured_shared_gb300 import padoc

from test_gpu_lm_loss import check, launch, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,D,V", [(700, 512, 9000), (3, 64, 20000)])
def test_wait_timeout_is_reported_and_recovered(padoc_lib, n, D, V):
    import torch
    h, w, t, d = make(n, D, V, seed=1, masked=0.1)
    t[0] = 0
    padoc.device_status()
    padoc.debug_set_wait_limit(1)
    try:
        launch(h, w, t, d)
        torch.cuda.synchronize()
        with pytest.raises(padoc.PadocError) as e:
            padoc.device_status()
        assert e.value.code == padoc.ERR_DEVICE_TIMEOUT
    finally:
        padoc.debug_set_wait_limit(0)
    padoc.device_status()
    want = reference(h, w, t, d)
    for _ in range(2):
        check(launch(h, w, t, d), *want)
