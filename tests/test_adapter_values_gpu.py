"""adapter_add at the edges of its values: a token without an adapter keeps the
bits of its row."""
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
