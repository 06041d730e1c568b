"""One adapter workspace for a server's largest batch serves every smaller one."""
import pytest
import torch

from parity_helpers import Guarded, dev

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def bl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_ternary_weight_b200 as b
    return b


def test_size_falls_neither_with_tokens_nor_with_rank(bl):
    def size(T, r):
        return bl.lib.bitlinear_adapter_workspace_bytes(T, r)

    sizes = torch.tensor([size(T, 16) for T in range(1, 12000)])
    assert (sizes.diff() >= 0).all() and sizes[0] > 0
    for T in (1, 31, 128, 129, 592, 4096, 9600, 1 << 20, (1 << 31) - 1):
        assert all(size(T, r) <= size(T, r + 8) for r in range(8, 128, 8))
    tall = [size(1 << e, 64) for e in range(31)]
    assert tall == sorted(tall)


@pytest.mark.parametrize("most,rank,T,r", [(4096, 16, 592, 16), (4096, 16, 526, 16), (9600, 16, 337, 16),
                                           (4096, 64, 1, 64), (600, 128, 129, 8), (2048, 24, 128, 16)])
def test_a_workspace_serves_fewer_tokens_and_lower_ranks(bl, most, rank, T, r):
    g = torch.Generator().manual_seed(T)
    K, N, n = 2560, 264, 5
    x, y = torch.randn(T, K, generator=g).to(BF16).to(dev()), torch.randn(T, N, generator=g).to(BF16).to(dev())
    down = (torch.randn(n, r, K, generator=g) * K ** -0.5).to(BF16).to(dev())
    up = (torch.randn(n, N, r, generator=g) * r ** -0.5).to(BF16).to(dev())
    index = torch.randint(-1, n, (T,), generator=g).to(torch.int32).to(dev())
    ws = Guarded(bl.adapter_workspace(most, rank, dev()).numel(), torch.uint8, dev())
    got = bl.adapter_add(y, x, down, up, index, workspace=ws.view)
    want = bl.adapter_add(y, x, down, up, index)
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0 and ws.intact()
    assert torch.equal(got, want) and not torch.equal(got, y)
