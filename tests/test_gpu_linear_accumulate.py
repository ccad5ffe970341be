"""The dense product's weight gradients, added to gradients that are there
already: one rounding at the size of the sum, which is that of
one fp32 addition of what the call writes where it does not add."""
import pytest

from tests.test_gpu_linear import _moe, _nan
from tests.test_linear_plan_host import LARGE

pytestmark = pytest.mark.gpu


# the large tiles, and the small ones in one slice, a few and many
@pytest.mark.parametrize("T,K,N", [s[:3] for s in LARGE] + [(700, 1088, 576), (1300, 512, 1408), (20011, 128, 192), (65600, 128, 256)])
def test_one_rounding_at_the_size_of_the_sum(T, K, N):
    import torch
    m = _moe()
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    dz, x = rand(T, N, std=0.1).bfloat16(), rand(T, K).bfloat16()
    old_w, old_b = rand(N, K, std=1e4), rand(N, std=1e4)
    ws = torch.empty(max(1, m.moe_linear_workspace_size(m.make_linear_shape(T, K, N))), dtype=torch.uint8, device="cuda")
    dw, db = _nan(N, K, dtype=torch.float32), _nan(N, dtype=torch.float32)
    print(f"[linear wgrad] added, T={T} K={K} N={N}", flush=True)
    m.moe_linear_wgrad(m.make_linear_shape(T, K, N, flags=m.MOE_LINEAR_OVERWRITE_DW), dz, x, dw, db, ws, ws.numel())
    got_w, got_b = old_w.clone(), old_b.clone()
    m.moe_linear_wgrad(m.make_linear_shape(T, K, N), dz, x, got_w, got_b, ws, ws.numel())
    assert torch.equal(got_w, old_w + dw) and torch.equal(got_b, old_b + db)
