"""Row lists are host memory that an upload copies: on a captured stream, whose
replays would read that memory again, an upload and an append_rope that needs
one are refused and change nothing; a write whose lists were uploaded before is
captured and replayed as documented."""
import gc

import numpy as np
import pytest

import i4ref
from tree_structured_shared_gb300 import padoc

from test_gpu_kv_rows import make_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
def test_lists_are_not_uploaded_into_a_graph(padoc_lib, request, dtype):
    import torch
    Hkv, n = 2, 16 * 230
    pool, kp, vp = make_pool(torch, 500, Hkv, dtype, max_bps=480)
    few, many, late = pool.alloc(0), pool.alloc(0), pool.alloc(20)
    k, v = (torch.randn(n, Hkv, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = np.arange(20, dtype=np.int32)[::-1].copy()
    rope = padoc.Rope(torch.from_numpy(i4ref.rope_table(300, 128)).cuda(), 128)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    rows, fresh = (padoc.KVRows(pool, [late], [0], [0, 20], positions=pos) for _ in range(2))
    rows.upload(ws, ws.numel())
    before, dirty = pool.stats(), [pool.seq_info(s) for s in (few, many, late)]
    torch.cuda.synchronize()
    codes = []

    def code(fn, *a, **kw):
        try:
            fn(*a, **kw)
        except padoc.PadocError as e:
            codes.append((e.code, "captured" in str(e)))
        else:
            codes.append(None)

    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    # an earlier test's pool that is collected now would free its block table, which ends a capture
    gc.collect()
    gc.disable()
    request.addfinalizer(gc.enable)
    with torch.cuda.graph(g, stream=st):
        code(pool.append_rope, [few], [0, 20], k, v, ws, ws.numel(), positions=pos, rope=rope)  # positions
        code(pool.append_rope, [many], [0, n], k, v, ws, ws.numel())                            # more than 224 blocks
        code(fresh.upload, ws, ws.numel())
        rows.write(k, v, ws, rope=rope)
    assert codes == [(padoc.ERR_INVALID, True)] * 3
    assert pool.stats() == before and [pool.seq_info(s) for s in (few, many, late)] == dirty
    # the captured write, and the refused calls outside a capture
    g.replay()
    pool.advance(late, 20)
    pool.append_rope([few], [0, 20], k, v, ws, ws.numel(), positions=pos, rope=rope)
    pool.append_rope([many], [0, n], k, v, ws, ws.numel())
    back = padoc.KVRows(pool, [late, few, many], [0, 0, 0], [0, 20, 40, 40 + n])
    ws2 = torch.empty(back.ws_size() + 16, dtype=torch.uint8, device="cuda")
    back.upload(ws2, ws2.numel())
    ko, vo = (torch.empty(back.n, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    back.gather(ko, vo, ws2)
    torch.cuda.synchronize()
    assert torch.equal(ko[:20], ko[20:40]) and torch.equal(vo[:20], vo[20:40])
    if dtype == padoc.BF16:
        assert torch.equal(ko[40:], k) and torch.equal(vo, torch.cat([v[:20], v[:20], v]))
    else:
        want = i4ref.stored(k.double().cpu().numpy(), v.double().cpu().numpy())
        assert np.array_equal(ko[40:].double().cpu().numpy(), want[0]) and np.array_equal(vo[40:].double().cpu().numpy(), want[1])
