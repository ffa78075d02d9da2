"""qkv_rope and kv_append: columns that are not turned stay, whatever stands beside them."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rope import Rows, w12  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot", [(128, 0), (128, 64), (96, 32), (256, 8), (72, 32)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["float", "bf16"])
def test_columns_that_are_not_turned(w12, d, rot, inter, kind):
    """Infinities, NaN and both zeros among the columns from rot_dim on: bit for bit what was there, rounded to bf16."""
    r = Rows(w12, d + rot, 9, 3, 2, d, rot, norm="", interleaved=inter, kind=kind)
    x = r.x.unflatten(1, (-1, d))[..., rot:]
    g = torch.Generator(device="cuda").manual_seed(1)
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0], device="cuda", dtype=r.x.dtype)
    put = torch.rand(x.shape, generator=g, device="cuda") < 0.2
    x.copy_(torch.where(put, odd[torch.randint(0, 5, x.shape, generator=g, device="cuda")], x))
    want = x.to(torch.bfloat16)
    got = torch.cat(w12.qkv_rope(r.x, r.form, r.pos), 1)[..., rot:]
    assert bool((got.isnan() == want.isnan()).all())
    same = got.contiguous().view(torch.int16) == want.contiguous().view(torch.int16)
    assert bool((same | want.isnan()).all())


def test_appended_columns_that_are_not_turned(w12):
    r = Rows(w12, 1, 5, 4, 2, 128, 64, norm="")
    x = r.x.unflatten(1, (-1, 128))
    x[:, 4:6, 100] = float("inf")
    kc, vc = [torch.zeros((2, 8, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w12.kv_append(r.x, r.form, r.pos, w12.KVCache(kc, vc), torch.arange(5, device="cuda"))
    assert torch.equal(kc.view(16, 2, 128)[:5, :, 64:], x[:, 4:6, 64:].to(torch.bfloat16))
