"""adapter_add at the edges of its values: a token without an adapter keeps the
bits of its row, and inner values at and beyond the end of fp32's range enter
the second product as what they are."""
import pytest
import torch

from parity_helpers import dev

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def bl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_ternary_weight_b200 as b
    return b


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else I32)


# few and many tokens (eight warps a tile, a tile, runs of tiles), rows of whole
# 16-byte vectors and others, every rank's kernel
@pytest.mark.parametrize("T,K,N,r,n", [(1, 64, 8, 8, 1), (5, 256, 333, 16, 3), (33, 128, 264, 40, 4),
                                       (300, 256, 1001, 64, 7), (4096, 64, 2560, 16, 9), (4096, 64, 1280, 128, 1),
                                       (700, 128, 640, 24, 600)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tokens_without_an_adapter_keep_their_bits(bl, T, K, N, r, n, dtype):
    """Every bit pattern of bf16 (fp32: with bits below), so both zeros,
    subnormals, infinities and NaNs with payloads, beside tokens that have an
    adapter and tokens whose adapter does not exist."""
    g = torch.Generator().manual_seed(T + N + r)
    high = torch.randint(0, 1 << 16, (T, N), generator=g)
    high[:, ::3] = 0x8000                                        # -0
    if dtype == BF16:
        y = high.to(torch.int16).view(BF16)
    else:
        y = torch.where(high == 0x8000, high << 16, (high << 16) + torch.randint(0, 1 << 16, (T, N), generator=g))
        y = y.to(I32).view(F32)
    index = torch.randint(-2, n + 1, (T,), generator=g).to(I32)
    index[0] = -1
    x = torch.randn(T, K, generator=g).to(BF16).to(dev())
    down, up = torch.randn(n, r, K, generator=g).to(BF16).to(dev()), torch.randn(n, N, r, generator=g).to(BF16).to(dev())
    kept = (index < 0) | (index >= n)
    yd, at = y.to(dev()), index.to(dev())
    got = bl.adapter_add(yd, x, down, up, at)
    torch.cuda.synchronize()
    assert bl.last_device_status() == (bl.BL_ERR_SHAPE if (index >= n).any() else 0)
    assert torch.equal(_bits(got.cpu())[kept], _bits(y)[kept])
    bl.adapter_add(yd, x, down, up, at, out=yd)
    torch.cuda.synchronize()
    bl.last_device_status()
    assert torch.equal(_bits(yd.cpu())[kept], _bits(y)[kept])
    assert torch.equal(_bits(yd), _bits(got))


@pytest.mark.parametrize("T,N", [(3, 40), (3, 37), (200, 264), (200, 75)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_inner_values_give_infinite_outputs(bl, T, N, dtype):
    """u = 2 * 2^127 is infinite in fp32: up u is +-inf by up's sign, not NaN.
    The other ranks' terms are finite and drop out of the sum."""
    g = torch.Generator().manual_seed(T + N)
    K, r = 64, 16
    x, down = torch.zeros(T, K), torch.randn(1, r, K, generator=g)
    x[:, 5:9] = torch.randn(T, 4, generator=g)
    x[:, 0], down[0, :, 0], down[0, 3, 0] = 2.0 ** 127, 0.0, 2.0
    up = torch.randn(1, N, r, generator=g).sign() * (0.5 + torch.rand(1, N, r, generator=g))
    y = torch.randn(T, N, generator=g).to(dtype)
    index = torch.zeros(T, dtype=I32)
    index[1] = -1
    got = bl.adapter_add(*(t.to(dev()) for t in (y, x.to(BF16), down.to(BF16), up.to(BF16), index))).cpu()
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0
    want = (up[0, :, 3].sign() * float("inf")).expand(T, N).to(dtype).clone()
    want[1] = y[1]
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,N", [(3, 40), (200, 75)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_inner_values_above_the_largest_bf16_stay_finite(bl, T, N, dtype):
    """u = 2^128 - 2^104 (fp32's largest value, as a sum of three products) lies
    above bf16's largest, 2^128 - 2^120, and would round to infinity; with up
    2^-120 the output is near 2^8.  u enters with 16 bits or more (2^-16 of it),
    the output's rounding adds 2^-8 or 2^-24."""
    K, r = 64, 8
    x, down = torch.zeros(T, K), torch.zeros(1, r, K)
    # 2^127 (1 + 127/128) + 2^119 (1 + 127/128) + 2^111 (1 + 127/128) = 2^128 - 2^104
    for j, e in enumerate((127, 119, 111)):
        x[:, j], down[0, :, j] = 2.0 ** (e - 100) * (255 / 128), 2.0 ** 100
    up = torch.full((1, N, r), 0.0)
    up[0, :, 1] = torch.where(torch.arange(N) % 2 == 0, 2.0 ** -120, -2.0 ** -120)
    y = torch.zeros(T, N, dtype=dtype)
    got = bl.adapter_add(*(t.to(dev()) for t in (y, x.to(BF16), down.to(BF16), up.to(BF16),
                                                 torch.zeros(T, dtype=I32)))).cpu().double()
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0
    want = (up[0, :, 1].double() * (2.0 ** 128 - 2.0 ** 104)).expand(T, N)
    tol = (2.0 ** -16 + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24)) * want.abs()
    assert ((got - want).abs() <= tol).all(), float((got - want).abs().max())
