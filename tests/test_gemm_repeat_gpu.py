"""The prefill GEMM gives the same sums every time, also where its first weight
tiles come late (from HBM, behind another kernel's writes)."""
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(8192, 2560, 6912), (2048, 6912, 2560)])
def test_gemm_repeats_exactly(M, N, K):
    import bit_ternary_weight_b200 as bl
    g = torch.Generator(device="cuda").manual_seed(M)
    w = bl.pack(torch.randn(N, K, device="cuda", generator=g))
    q, d, r = bl.quantize_act(torch.randn(M, K, device="cuda", generator=g).bfloat16())
    acc = torch.empty(M, N, dtype=torch.int32, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    # |sum| <= 128 K < 2^53: the products of doubles are exact
    codes = torch.from_numpy(oracle.unpack(w.packed.cpu().numpy(), N, K)).to("cuda").double()
    want = torch.empty_like(acc)
    for i in range(0, M, 1024):
        want[i:i + 1024] = (q[i:i + 1024].double() @ codes.T).int()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1500):
        acc.fill_(-1)
        bl.gemm(w, q, d, r, out=y, acc_dbg=acc)
        wrong += (acc != want).sum()
    assert int(wrong) == 0
    assert bl.last_device_status() == 0
