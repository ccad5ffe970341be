"""The dense product and its gradients on every kernel that runs them, named by
the record of the launches, so that a rule that changes cannot empty a test.

Besides the operators' own bars (test_gpu_linear.py), which grow with the
length of a sum as its worst case does, the sums here are exact: small whole
numbers, whose fp32 sums below 2^24 have no rounding in any order, so that a
term lost or taken twice, or a slice, shows as a difference; y and dx are then
one rounding to bf16 of an exact number, and have to be equal too.
"""
import pytest

from tests import test_gpu_linear as base
from tests.launched import assert_launched
from tests.test_linear_plan_host import LARGE

pytestmark = pytest.mark.gpu

TILE = "ffn_tile_kernel<false, "
WIDE, FEW = "linear_wide_kernel<", "ffn_few_kernel<false, "
# kernel by kernel, sums of several stages, rows and columns that leave tiles partly empty: T, K, N and the launches
FORWARD = [
    ((100, 1088, 4160), (FEW + "2, 3, 4, 3>",)),
    ((20, 576, 16448), (FEW + "2, 2, 8, 3>",)),
    ((1, 576, 65536), (FEW + "1, 1, 4, 3>",)),
    ((300, 1088, 2112), (TILE + "64, 64, 32, 64, 4, 2, false, 3>",)),
    ((1000, 1984, 1408), (TILE + "64, 128, 32, 64, 2, 3, false, 3>",)),
    ((1500, 1088, 2112), (TILE + "128, 128, 64, 64, 2, 2, false, 3>",)),
    ((1580, 1088, 2496), (TILE + "64, 128, 32, 64, 1, 3, false, 3>",)),
    ((2100, 1088, 2112), (TILE + "128, 128, 64, 64, 1, 2, false, 3>",)),
    ((4200, 1088, 2112), (WIDE + "false, ",)),
    ((12400, 1088, 1984), (WIDE + "false, ",)),
    ((8300, 576, 2112), (WIDE + "false, ", TILE + "128, 128, 64, 64, 2, 2, false, 3>")),
]
DGRAD = [
    ((1000, 1984, 1408), (TILE + "64, 128, 32, 64, 2, 2, true, 4>",)),
    ((1100, 1984, 1408), (TILE + "128, 128, 64, 64, 2, 2, true, 4>",)),
    ((4200, 1088, 2112), (TILE + "128, 128, 64, 64, 1, 2, true, 4>",)),
    ((5000, 2112, 2112), (WIDE + "true, ",)),
    ((12400, 1984, 1088), (WIDE + "true, ",)),
    ((9001, 2112, 1088), (WIDE + "true, ", TILE + "128, 128, 64, 64, 2, 2, true, 4>")),
    ((700, 1088, 576), ("linear_few_dx_kernel<64, 3>",)),
    ((300, 1088, 1088), ("linear_few_dx_kernel<32, 3>",)),
]


def _whole(gen, *shape, most=2):
    """Whole numbers from -most to most."""
    import torch
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").bfloat16()


def _exact(v):
    """An fp64 result as the kernels' fp32 sums hold it: whole, below 2^24."""
    assert float(v.abs().max()) < 2 ** 24
    return v.float()


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("shape,launches", FORWARD)
def test_forward(shape, launches):
    import torch
    m = base._moe()
    T, K, N = shape
    gen = _gen(T + K + N)
    x, w, b, res = _whole(gen, T, K), _whole(gen, N, K), _whole(gen, N, most=50), _whole(gen, T, N, most=100)
    prod = x.double() @ w.double().t()
    print(f"[linear] whole numbers T={T} K={K} N={N}", flush=True)
    for act, bias, r in (("none", b, res), ("relu", b, None), ("relu", None, res), ("none", None, None)):
        s = m.make_linear_shape(T, K, N, act=base.ACTS.index(act))
        z, y = base._nan(T, N), base._nan(T, N)
        assert_launched(lambda: m.moe_linear_fwd(s, x, w, bias, r, z, y), *launches)
        z64 = prod if bias is None else prod + bias.double()
        y64 = z64.clamp(min=0) if act == "relu" else z64
        y64 = y64 if r is None else y64 + r.double()
        assert torch.equal(z, _exact(z64).bfloat16()) and torch.equal(y, _exact(y64).bfloat16())


@pytest.mark.parametrize("shape", [s for s, _ in FORWARD if s[0] * s[1] * s[2] < 2 * 10 ** 10])
def test_forward_against_the_oracle(shape):
    base.test_forward(*shape)


@pytest.mark.parametrize("shape,launches", DGRAD)
def test_dgrad(shape, launches):
    import torch
    m = base._moe()
    T, K, N = shape
    gen = _gen(T + K + N + 1)
    dz, w, add = _whole(gen, T, N), _whole(gen, N, K), _whole(gen, T, K, most=100)
    z = _whole(gen, T, K)
    prod = dz.double() @ w.double()
    s = m.make_linear_shape(T, K, N)
    print(f"[linear dgrad] whole numbers T={T} K={K} N={N}", flush=True)
    for act, a in ((None, add), ("relu", None), ("relu", add), (None, None)):
        dx = base._nan(T, K)
        call = lambda: m.moe_linear_dgrad(s, dz, w, z if act else None, base.ACTS.index(act or "none"), a, dx)  # noqa: E731
        assert_launched(call, *launches)
        dx64 = prod * (z.double() > 0) if act else prod
        assert torch.equal(dx, _exact(dx64 if a is None else dx64 + a.double()).bfloat16())


@pytest.mark.parametrize("shape", [s for s, _ in DGRAD if s[0] * s[1] * s[2] < 25 * 10 ** 9])
def test_dgrad_against_the_oracle(shape):
    base.test_dgrad(*shape)


# the large tiles, and the small ones in no, a few and many slices, the last of them of a few tokens
@pytest.mark.parametrize("T,K,N,slices", LARGE + [(700, 1088, 576, 0), (1300, 512, 1408, 0), (65600, 128, 256, 0),
                                                  (20011, 128, 192, 0), (3001, 64, 64, 0), (1, 2048, 1408, 0)])
def test_wgrad(T, K, N, slices):
    """slices: of the large tiles, 0 for the small ones."""
    import torch
    m = base._moe()
    gen = _gen(T + K + N + 2)
    dz, x = _whole(gen, T + 3, N), _whole(gen, T + 3, K)
    dz[T:], x[T:] = float("nan"), float("nan")  # rows behind the last token
    dw64, db64 = dz[:T].double().t() @ x[:T].double(), dz[:T].double().sum(0)
    acc, over = m.make_linear_shape(T, K, N), m.make_linear_shape(T, K, N, flags=m.MOE_LINEAR_OVERWRITE_DW)
    ws = torch.full((max(1, m.moe_linear_workspace_size(acc)),), 0xFF, dtype=torch.uint8, device="cuda")
    print(f"[linear wgrad] whole numbers T={T} K={K} N={N}", flush=True)

    def run(shape, dw, db):
        call = lambda: m.moe_linear_wgrad(shape, dz, x, dw, db, ws, ws.numel())  # noqa: E731
        if slices == 1:
            assert_launched(call, "linear_dw_kernel<true>" if shape is acc else "linear_dw_kernel<false>")
        elif slices:
            assert_launched(call, "linear_dw_kernel<false>", "linear_dw_reduce_kernel")
        else:
            call()
    for with_db in (True, False):
        dw, db = base._nan(N, K, dtype=torch.float32), base._nan(N, dtype=torch.float32)
        run(over, dw, db if with_db else None)
        assert torch.equal(dw, _exact(dw64))
        assert torch.equal(db, _exact(db64)) if with_db else torch.isnan(db).all()
        old_w, old_b = _whole(gen, N, K, most=100).float(), _whole(gen, N, most=100).float()
        dw, db = old_w.clone(), old_b.clone()
        run(acc, dw, db if with_db else None)
        assert torch.equal(dw, _exact(dw64 + old_w.double()))
        assert torch.equal(db, _exact(db64 + old_b.double()) if with_db else old_b)


@pytest.mark.parametrize("T,K,N", [s[:3] for s in LARGE])
def test_wgrad_against_the_oracle(T, K, N):
    base.test_wgrad(T, K, N)


@pytest.mark.parametrize("T,K,N", [(65, 65536, 64), (300, 65536, 1088), (17, 64, 16448)])
def test_long_sums_lose_no_term(T, K, N):
    """The longest sums of the forward and of the input gradient."""
    import torch
    m = base._moe()
    gen = _gen(K)
    x, w = _whole(gen, T, K), _whole(gen, N, K)
    y = base._nan(T, N)
    print(f"[linear] whole numbers T={T} K={K} N={N}", flush=True)
    m.moe_linear_fwd(m.make_linear_shape(T, K, N), x, w, None, None, None, y)
    assert torch.equal(y, _exact(x.double() @ w.double().t()).bfloat16())
    wt, dx = w.t().contiguous(), base._nan(T, N)  # [K, N]: the sum of dx runs over K
    m.moe_linear_dgrad(m.make_linear_shape(T, N, K), x, wt, None, m.MOE_ACT_NONE, None, dx)
    assert torch.equal(dx, y)
