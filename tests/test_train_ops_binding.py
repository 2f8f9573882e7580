"""What the Python binding of the operators around the attention of a training step refuses by
the tensors' types, sizes and layouts, which the library cannot see.  On the CPU, without the
library: every refusal comes before it is called."""
import pytest

from tree_structured_shared_gb300 import padoc

torch = pytest.importorskip("torch")


def refused(f, *a, **kw):
    with pytest.raises(padoc.PadocError) as e:
        f(*a, **kw)
    assert e.value.code == padoc.ERR_INVALID


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(padoc, "_lib", None)
    monkeypatch.setattr(padoc, "lib", lambda: pytest.fail("the library was called"))


@pytest.fixture
def head():
    return padoc.LmLoss(torch.zeros(6, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16),
                        torch.zeros(6, dtype=torch.int32))


WS = torch.empty(1 << 16, dtype=torch.uint8)
BAD_ROWS = [torch.zeros(6, dtype=torch.bfloat16), torch.zeros(6, dtype=torch.float64), torch.zeros(5),
            torch.zeros(12)[::2], torch.ones(()).expand(6), torch.zeros(6, 2)[:, 0], torch.zeros(6, device="meta")]


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_loss_rows(head, i):
    bad, good = BAD_ROWS[i], torch.zeros(6)
    g = torch.zeros(6, 64, dtype=torch.bfloat16)
    refused(head.forward, bad, good, WS, WS.numel())
    refused(head.forward, good, bad, WS, WS.numel())
    refused(head.backward, bad, good, g, None, WS, WS.numel())
    refused(head.backward, good, bad, g, None, WS, WS.numel())


def test_expanded_gradient_of_a_mean(head):
    """What autograd hands on for the mean of the losses: one value, expanded."""
    loss = torch.zeros(6, requires_grad=True)
    seen = []
    loss.register_hook(seen.append)
    loss.sum().backward()
    assert seen[0].stride() == (0,)
    refused(head.backward, torch.zeros(6), seen[0], None, torch.zeros(9, 64, dtype=torch.bfloat16), WS, WS.numel())


@pytest.mark.parametrize("which", ["dh", "dw"])
def test_loss_gradients(head, which):
    rows = 6 if which == "dh" else 9
    bf = dict(dtype=torch.bfloat16)
    for bad in (torch.zeros(rows, 64), torch.zeros(rows, 64, dtype=torch.float16), torch.zeros(rows, 72, **bf)[:, :64],
                torch.zeros(64, rows, **bf).T, torch.zeros(rows - 1, 64, **bf), torch.zeros(rows, 64, device="meta", **bf)):
        a = dict(dh=None, dw=None)
        a[which] = bad
        refused(head.backward, torch.zeros(6), torch.zeros(6), a["dh"], a["dw"], WS, WS.numel())


def test_workspace(head):
    f = torch.zeros(6)
    refused(head.forward, f, f.clone(), WS, WS.numel() + 1)
    refused(head.forward, f, f.clone(), WS[::2], WS.numel() // 2)
    refused(head.backward, f, f, None, torch.zeros(9, 64, dtype=torch.bfloat16), WS[:100], 101)


def test_inputs_on_one_device():
    h, w, t = torch.zeros(6, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(6, dtype=torch.int32)
    for i in range(3):
        a = [h, w, t]
        a[i] = a[i].to("meta")
        refused(padoc.LmLoss, *a)


def rope(x, out, H=2, d=64, n=6, **kw):
    padoc.rope_apply(padoc.Rope(4096, 64, n_pos=100), n, d, x, out, H, **kw)


def test_rope_rows():
    bf = dict(dtype=torch.bfloat16)
    x, out = torch.zeros(6, 128, **bf), torch.zeros(6, 2, 64, **bf)
    i32 = torch.zeros(6, dtype=torch.int32)
    f32 = x.float()
    for bad in (f32, x[:5], torch.zeros(6, 128, dtype=torch.float16), torch.zeros(6, 256, **bf)[:, ::2], torch.zeros(128, 6, **bf).T,
                torch.zeros(6, 2, 72, **bf)[..., :64], torch.zeros(2, 3, 256, **bf)[..., :128]):
        refused(rope, bad, out)
        refused(rope, x, bad)
        refused(rope, x, out, k=bad, k_out=out.clone(), Hkv=2)
        refused(rope, x, out, k=x.clone(), k_out=bad, Hkv=2)
    refused(rope, f32, out, q_stride=128)               # a stride does not change the type
    refused(rope, x[:5], out, q_stride=128)
    refused(rope, x, out, dtype=padoc.F32)
    for bad in (i32.long(), i32[:5], torch.zeros(12, dtype=torch.int32)[::2]):
        refused(rope, x, out, positions=bad)


def test_rope_table():
    for bad in (torch.zeros(10, 64, dtype=torch.float64), torch.zeros(9, 64), torch.zeros(10, 128)[:, :64]):
        refused(padoc.rope_table, bad, 10, 64, 1.0e4)


@pytest.mark.parametrize("make,stride", [
    (lambda x: x, 256), (lambda x: x[:, :128], 256), (lambda x: x.view(6, 4, 64)[:, :2], 256), (lambda x: x[:, :128].contiguous(), 128),
    (lambda x: x[:, :128].reshape(12, 64), 128), (lambda x: x[:, :128].reshape(-1), 128), (lambda x: x[:, :128].reshape(2, 3, 2, 64).contiguous(), 128),
    (lambda x: torch.cat([x, x])[:, :128], 256), (lambda x: x.data_ptr(), 128), (lambda x: torch.cat([x, x])[:, :128].contiguous(), 128)])
def test_rope_strides_of_tensors(make, stride):
    """The rows that a call without strides takes."""
    x = torch.zeros(6, 256, dtype=torch.bfloat16)
    y = make(x)
    assert padoc._rows(y, 6, 128, 6 * 256, None, torch.bfloat16) == (y if isinstance(y, int) else y.data_ptr(), stride)
    assert padoc._rows(y, 6, 128, 6 * 256, 264, torch.bfloat16)[1] == 264
