"""Prompt operators on the GPU against their definitions in 64 bits: per-head
norm + rotation + cache append, causal attention of packed sequences, and
low-rank adapters; the sizes, strides and masks where each can go wrong, and a
run of them together.

Tolerances, from the arithmetic (u8 = 2^-8 is half a bf16 step, u24 = 2^-24
half an fp32 step, both relative):
  rope     one rounding to bf16 after fp32 arithmetic on values of the pair's
           size: u8 |y| + 16 u24 (|a| + |b|) (a norm's 128-term mean square in
           fp32 is off by at most 24 u24 in a tree of 16 + 3 additions, its
           root by half of that).  Without a norm the two sides are equal.
  attention  each weight is rounded to bf16 (u8) and evaluated to 2^-12 (the
           exponential, and scores of fp32 sums: 128 terms of products that
           are exact, 2^-23 each, far below that for the sizes here), so a sum
           of w_j V_j over w is off by at most (u8 + 2 * 2^-12) sum w_j |V_j|;
           the output's rounding adds u8 |out|.
  adapter  the r values between the products enter the second with 16 bits
           (2^-16 relative) after sums of K exact products (K 2^-23 of the sum
           of magnitudes), the second sum has 2 r terms (2^-23 each); the
           output's rounding adds u8 or u24 of |out|.
"""
import numpy as np
import pytest
import torch

import oracle
from parity_helpers import Guarded, dev

pytestmark = pytest.mark.gpu

D = 128
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U8, U24 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def bl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_ternary_weight_b200 as b
    return b


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _within(got, want, tol, name="output"):
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    err = (got - want).abs()
    bad = err > tol
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside; worst {float((err - tol).max()):.3g} "
                           f"over at {int((err - tol).argmax())}")


def _clean(bl):
    torch.cuda.synchronize()
    assert bl.last_device_status() == 0


# ------------------------------------------------------------------ attention

def _attention64(q, k, v, cu_q, cu_k, scale=D ** -0.5):
    """out and sum_j w_j |V_j| in fp64; rows of no sequence are NaN."""
    Tq, H = q.shape[:2]
    G = H // k.shape[1]
    out = torch.full((Tq, H, D), float("nan"), dtype=torch.float64)
    mag = torch.zeros(Tq, H, D, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        m, n = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        qs, ks, vs = q[cu_q[b]:cu_q[b + 1]].double(), k[cu_k[b]:cu_k[b + 1]].double(), v[cu_k[b]:cu_k[b + 1]].double()
        for i in range(m):
            seen = max(0, i + n - m + 1)
            for h in range(H):
                if seen == 0:
                    out[cu_q[b] + i, h] = 0
                    continue
                w = torch.softmax(scale * (ks[:seen, h // G] @ qs[i, h]), 0)
                out[cu_q[b] + i, h] = w @ vs[:seen, h // G]
                mag[cu_q[b] + i, h] = w @ vs[:seen, h // G].abs()
    return out, mag


def _attention_fast64(q, k, v, cu_q, cu_k, scale=D ** -0.5):
    """The same for finite inputs, a head of a sequence at a time."""
    Tq, H = q.shape[:2]
    G = H // k.shape[1]
    out = torch.full((Tq, H, D), float("nan"), dtype=torch.float64)
    mag = torch.zeros(Tq, H, D, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        m, n = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        future = torch.ones(m, n, dtype=torch.bool).triu(n - m + 1)
        for h in range(H):
            s = scale * (q[cu_q[b]:cu_q[b + 1], h].double() @ k[cu_k[b]:cu_k[b + 1], h // G].double().t())
            w = torch.softmax(s.masked_fill(future, -float("inf")), -1).nan_to_num(0.0)
            vs = v[cu_k[b]:cu_k[b + 1], h // G].double()
            out[cu_q[b]:cu_q[b + 1], h] = w @ vs
            mag[cu_q[b]:cu_q[b + 1], h] = w @ vs.abs()
    return out, mag


def _cu(lens, start=0):
    out = [start]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _check_attention(bl, got, q, k, v, cu_q, cu_k, scale=D ** -0.5, fill=None):
    _clean(bl)
    want, mag = _attention_fast64(q, k, v, cu_q, cu_k, scale)
    mine = ~want.isnan()
    tol = (U8 + 2 * 2.0 ** -12) * mag + U8 * want.nan_to_num(0.0).abs()
    _within(got.cpu()[mine], want[mine], tol[mine])
    if fill is not None:
        assert (got.cpu()[~mine] == fill).all(), "rows of no sequence were written"


def _rand(g, *shape, s=1.0):
    return (s * torch.randn(*shape, generator=g)).to(BF16)


def _on_dev(cu):
    return torch.tensor(cu, dtype=I32, device=dev())


LAYOUTS = [(20, 5), (16, 2), (8, 8), (7, 1), (6, 2), (64, 1), (3, 3)]


@pytest.mark.parametrize("H,Hkv", LAYOUTS)
@pytest.mark.parametrize("lens", [[1], [37], [128, 1, 127, 129], [0, 5, 0, 300, 2, 0], [64, 65, 63, 513]])
def test_prompts(bl, H, Hkv, lens):
    g = _gen(sum(lens) * 100 + H)
    cu = _cu(lens)
    T = cu[-1]
    q, k, v = _rand(g, T, H, D), _rand(g, T, Hkv, D, s=1.5), _rand(g, T, Hkv, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu))
    _check_attention(bl, out, q, k, v, cu, cu)


@pytest.mark.parametrize("H,Hkv", [(20, 5), (16, 2), (8, 8)])
@pytest.mark.parametrize("nq,nk", [([1] * 9, [1, 2, 127, 128, 129, 500, 1000, 3, 64]), ([1], [4097]),
                                   ([1, 4, 2, 1], [4000, 4, 131, 1]), ([100], [1100]), ([77, 300], [2000, 300]),
                                   ([1] * 200, [1 + (i * 37) % 300 for i in range(200)])])
def test_queries_behind_a_past(bl, H, Hkv, nq, nk):
    g = _gen(sum(nk) + H)
    cu_q, cu_k = _cu(nq), _cu(nk)
    q, k, v = _rand(g, cu_q[-1], H, D), _rand(g, cu_k[-1], Hkv, D, s=1.5), _rand(g, cu_k[-1], Hkv, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k))
    _check_attention(bl, out, q, k, v, cu_q, cu_k)


@pytest.mark.parametrize("H,Hkv,T", [(20, 5, 2100), (4, 1, 4500)])
def test_long_prompt(bl, H, Hkv, T):
    g = _gen(T)
    q, k, v = _rand(g, T, H, D), _rand(g, T, Hkv, D, s=1.5), _rand(g, T, Hkv, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev([0, T]))
    _check_attention(bl, out, q, k, v, [0, T], [0, T])


@pytest.mark.parametrize("H,Hkv,nq,nk", [(7, 1, [1400, 37, 300], None), (6, 2, [1400, 37, 300], None),
                                         (3, 3, [2500, 1400], None), (20, 5, [400, 300], [1000, 300]),
                                         (20, 5, [900, 60], [500, 1300]), (16, 2, [333] * 5, [333] * 5),
                                         (20, 5, [40] * 30, [40] * 30), (64, 1, [50, 90], [50, 800])])
def test_many_rows(bl, H, Hkv, nq, nk):
    """Enough rows that two tiles share a pass over the keys: groups that do
    not divide a tile, tiles that end inside a pair, queries before the keys."""
    g = _gen(sum(nq) + H)
    cu_q = _cu(nq)
    cu_k = _cu(nk or nq)
    q, k, v = _rand(g, cu_q[-1], H, D), _rand(g, cu_k[-1], Hkv, D, s=1.5), _rand(g, cu_k[-1], Hkv, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k))
    _check_attention(bl, out, q, k, v, cu_q, cu_k)


@pytest.mark.parametrize("H,Hkv,nq,nk", [(20, 5, 130, 9000), (8, 8, 40, 12000), (20, 5, 700, 7000)])
def test_few_rows_cut_into_many_parts(bl, H, Hkv, nq, nk):
    g = _gen(nq + nk)
    q, k, v = _rand(g, nq, H, D), _rand(g, nk, Hkv, D, s=1.5), _rand(g, nk, Hkv, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev([0, nq]), _on_dev([0, nk]))
    _check_attention(bl, out, q, k, v, [0, nq], [0, nk])


def test_one_token_on_a_very_long_cache(bl):
    g = _gen(5)
    n = 32768
    q, k, v = _rand(g, 1, 16, D), _rand(g, n, 2, D, s=1.5), _rand(g, n, 2, D)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev([0, 1]), _on_dev([0, n - 3]))
    _check_attention(bl, out, q, k, v, [0, 1], [0, n - 3])


@pytest.mark.parametrize("nq,nk", [([5, 3, 40], [2, 0, 40]), ([200], [70]), ([1, 1], [0, 0]), ([300, 1], [299, 0])])
def test_queries_that_see_nothing_get_zeros(bl, nq, nk):
    """More queries than keys, and no keys at all."""
    g = _gen(9)
    H, Hkv = 20, 5
    cu_q, cu_k = _cu(nq), _cu(nk)
    rows = max(1, cu_k[-1])
    q, k, v = _rand(g, cu_q[-1], H, D), _rand(g, rows, Hkv, D), _rand(g, rows, Hkv, D)
    out = torch.full((cu_q[-1], H, D), 7.0, dtype=BF16, device=dev())
    bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k), out=out)
    _check_attention(bl, out, q, k, v, cu_q, cu_k)
    for b in range(len(nq)):
        blind = max(0, nq[b] - nk[b])
        assert (out[cu_q[b]:cu_q[b] + blind] == 0).all()


def test_rows_of_no_sequence_stay(bl):
    """Rows in front of the first and behind the last sequence."""
    g = _gen(11)
    H, Hkv = 16, 2
    cu_q, cu_k = [3, 10, 10, 75], [6, 30, 200, 420]
    q, k, v = _rand(g, 90, H, D), _rand(g, 450, Hkv, D), _rand(g, 450, Hkv, D)
    out = torch.full((90, H, D), 7.0, dtype=BF16, device=dev())
    bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k), out=out)
    _check_attention(bl, out, q, k, v, cu_q, cu_k, fill=7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("nq,nk", [([1, 130, 1], [200, 130, 77]), ([700], [700]), ([40, 9], [40, 9])])
def test_what_no_query_sees_has_no_effect(bl, bad, nq, nk):
    """NaN and infinities around the sequences' keys: between them, behind the
    last one, and in keys and values that lie in a query's future."""
    g = _gen(13)
    H, Hkv, gap = 20, 5, 7
    starts = []
    at = gap
    for n in nk:
        starts.append(at)
        at += n + gap
    q = _rand(g, sum(nq), H, D)
    k, v = _rand(g, at, Hkv, D, s=1.5), _rand(g, at, Hkv, D)
    cu_q = _cu(nq)
    for b in range(len(nq)):      # one call each: key rows with gaps between the sequences
        kb, vb = torch.full_like(k, bad), torch.full_like(v, bad)
        s = slice(starts[b], starts[b] + nk[b])
        kb[s], vb[s] = k[s], v[s]
        qb = q[cu_q[b]:cu_q[b + 1]]
        out = bl.attention_prefill(qb.to(dev()), kb.to(dev()), vb.to(dev()), _on_dev([0, nq[b]]),
                                   _on_dev([s.start, s.stop]))
        _check_attention(bl, out, qb, k[s], v[s], [0, nq[b]], [0, nk[b]])
        if nq[b] > 1:             # the last key is seen by the last query alone
            kb[s.stop - 1], vb[s.stop - 1] = bad, bad
            out = bl.attention_prefill(qb.to(dev()), kb.to(dev()), vb.to(dev()), _on_dev([0, nq[b]]),
                                       _on_dev([s.start, s.stop]))
            want, mag = _attention_fast64(qb[:-1], k[s][:-1], v[s][:-1], [0, nq[b] - 1], [0, nk[b] - 1])
            _within(out.cpu()[:-1], want, (U8 + 2 * 2.0 ** -12) * mag + U8 * want.abs())


@pytest.mark.parametrize("nq,nk", [([150], [150]), ([1, 2, 1], [300, 2, 64]), ([513], [900])])
def test_strides(bl, nq, nk):
    """A cache [Hkv, rows, D], parts of a fused projection, padded heads."""
    g = _gen(17)
    H, Hkv = 20, 5
    cu_q, cu_k = _cu(nq), _cu(nk)
    Tq, Tk = cu_q[-1], cu_k[-1]
    qkv = _rand(g, Tq, H + 2 * Hkv, D).to(dev())
    cache = _rand(g, 2, Hkv, Tk + 31, D + 24).to(dev())
    q = qkv[:, :H]
    k, v = cache[0, :, :, 8:D + 8].transpose(0, 1), cache[1, :, :, 16:D + 16].transpose(0, 1)
    out = torch.full((H, Tq, D + 8), 7.0, dtype=BF16, device=dev())
    bl.attention_prefill(q, k, v, _on_dev(cu_q), _on_dev(cu_k), out=out[..., :D].transpose(0, 1))
    _check_attention(bl, out[..., :D].transpose(0, 1), q.cpu(), k.cpu(), v.cpu(), cu_q, cu_k)
    assert (out[..., D:] == 7.0).all()


@pytest.mark.parametrize("scale", [1.0, 1e-3, 30.0])
def test_scales_and_large_scores(bl, scale):
    """Scores from nearly equal to one that takes all, rising and falling with the key."""
    g = _gen(19)
    H, Hkv, T = 8, 2, 400
    q, k, v = _rand(g, T, H, D), _rand(g, T, Hkv, D), _rand(g, T, Hkv, D)
    ramp = torch.linspace(0, 2, T)[:, None, None]
    # score sums over 128 exact products: |s| up to about 1500 at scale 30 would cost bits
    q, k = (q * 0.25).to(BF16), (k * 0.25 + ramp * 0.25 * torch.tensor([1.0, -1.0])[None, :, None]).to(BF16)
    out = bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev([0, T]), scale=scale)
    _check_attention(bl, out, q, k, v, [0, T], [0, T], scale)


def test_bad_sequence_bounds_are_reported_and_write_nothing(bl):
    g = _gen(23)
    H, Hkv = 8, 2
    q, k, v = _rand(g, 40, H, D), _rand(g, 60, Hkv, D), _rand(g, 60, Hkv, D)
    for cu_q, cu_k, fine in [([0, 10, 41], [0, 30, 60], [0]), ([0, 10, 40], [0, 30, 61], [0]),
                             ([0, 10, 40], [0, 30, 20], [0]), ([-1, 10, 40], [0, 30, 60], [1]),
                             ([0, 20, 10], [0, 30, 60], [0])]:
        out = torch.full((40, H, D), 7.0, dtype=BF16, device=dev())
        bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k), out=out)
        torch.cuda.synchronize()
        assert bl.last_device_status() == bl.BL_ERR_SHAPE, (cu_q, cu_k)
        mine = torch.zeros(40, dtype=torch.bool)
        for b in fine:
            a, e = cu_q[b:b + 2]
            mine[a:e] = True
            want, mag = _attention_fast64(q[a:e], k[cu_k[b]:cu_k[b + 1]], v[cu_k[b]:cu_k[b + 1]], [0, e - a],
                                          [0, cu_k[b + 1] - cu_k[b]])
            _within(out[a:e], want, (U8 + 2 * 2.0 ** -12) * mag + U8 * want.abs())
        assert (out.cpu()[~mine] == 7.0).all(), (cu_q, cu_k)
    assert bl.last_device_status() == 0


def test_attention_writes_inside_its_buffers(bl):
    g = _gen(29)
    for H, Hkv, nq, nk in [(20, 5, [1, 33], [90, 200]), (16, 2, [129], [129])]:
        cu_q, cu_k = _cu(nq), _cu(nk)
        q, k, v = _rand(g, cu_q[-1], H, D), _rand(g, cu_k[-1], Hkv, D), _rand(g, cu_k[-1], Hkv, D)
        out = Guarded(cu_q[-1] * H * D, BF16, dev())
        ws = Guarded(bl.attention_prefill_workspace(H, Hkv, dev()).numel(), torch.uint8, dev())
        bl.attention_prefill(q.to(dev()), k.to(dev()), v.to(dev()), _on_dev(cu_q), _on_dev(cu_k),
                             out=out.view.view(-1, H, D), workspace=ws.view)
        _check_attention(bl, out.view.view(-1, H, D), q, k, v, cu_q, cu_k)
        assert out.intact() and ws.intact()


def test_attention_graph_replays_and_streams(bl):
    """One captured call replayed for other lengths and inputs in its buffers,
    and calls on two streams with a workspace each."""
    g = _gen(31)
    H, Hkv = 20, 5
    Tq, Tk, B = 6, 900, 3
    q, k, v = (torch.zeros(Tq, H, D, dtype=BF16, device=dev()), torch.zeros(Tk, Hkv, D, dtype=BF16, device=dev()),
               torch.zeros(Tk, Hkv, D, dtype=BF16, device=dev()))
    cq, ck = _on_dev([0, 1, 2, 3]), _on_dev([0, 1, 2, 3])
    out = torch.zeros(Tq, H, D, dtype=BF16, device=dev())
    ws = bl.attention_prefill_workspace(H, Hkv, dev())
    bl.attention_prefill(q, k, v, cq, ck, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.attention_prefill(q, k, v, cq, ck, out=out, workspace=ws)
    for nq, nk in [([1, 1, 1], [300, 5, 400]), ([2, 3, 1], [2, 3, 895]), ([0, 6, 0], [0, 900, 0])]:
        cu_q, cu_k = _cu(nq), _cu(nk)
        hq, hk, hv = _rand(g, Tq, H, D), _rand(g, Tk, Hkv, D), _rand(g, Tk, Hkv, D)
        q.copy_(hq), k.copy_(hk), v.copy_(hv), cq.copy_(torch.tensor(cu_q)), ck.copy_(torch.tensor(cu_k))
        out.fill_(7.0)
        graph.replay()
        _check_attention(bl, out, hq, hk, hv, cu_q, cu_k, fill=7.0)
    hq, hk, hv = _rand(g, 700, H, D), _rand(g, 700, Hkv, D), _rand(g, 700, Hkv, D)
    dq, dk, dv = hq.to(dev()), hk.to(dev()), hv.to(dev())
    cu = _on_dev([0, 1, 700])
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(3):
                o = bl.attention_prefill(dq, dk, dv, cu)
            outs.append(o)
    torch.cuda.synchronize()
    _check_attention(bl, outs[0], hq, hk, hv, [0, 1, 700], [0, 1, 700])
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_attention_same_bits_again(bl):
    g = _gen(37)
    q, k, v = (_rand(g, 300, h, D).to(dev()) for h in (20, 5, 5))
    one = _rand(g, 3, 20, D).to(dev())
    for args in [(q, k, v, _on_dev([0, 300])), (one, k, v, _on_dev([0, 1, 2, 3]), _on_dev([0, 90, 95, 300]))]:
        a = bl.attention_prefill(*args)
        for _ in range(5):
            assert torch.equal(a, bl.attention_prefill(*args))


# ------------------------------------------------------------------ norm + rotation + append

def _rope64(x, gain, eps, cs, halves):
    """The rotated heads in fp64 and |a| + |b| of each pair."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * gain.double()
    c, s = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    if halves:
        a, b = x[..., :64], x[..., 64:]
        return torch.cat([a * c - b * s, a * s + b * c], -1), torch.cat([a.abs() + b.abs()] * 2, -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return (torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2),
            torch.stack([a.abs() + b.abs()] * 2, -1).flatten(-2))


@pytest.mark.parametrize("T,H,Hkv", [(1, 20, 5), (1, 1, 1), (3, 16, 2), (33, 7, 1), (257, 20, 5), (1000, 3, 3)])
@pytest.mark.parametrize("dtype,gdtype,halves", [(BF16, BF16, False), (BF16, F32, True), (F32, F32, False),
                                                 (F32, BF16, True)])
def test_qk_norm_rope(bl, T, H, Hkv, dtype, gdtype, halves):
    g = _gen(T * 10 + H)
    P, R = T + 50, T + 9
    q, k, v = (torch.randn(T, h, D, generator=g).mul(3).to(dtype) for h in (H, Hkv, Hkv))
    k[T // 2] = 0                # a head of zeros: only eps keeps its norm finite
    qg, kg = ((1 + 0.2 * torch.randn(D, generator=g)).to(gdtype) for _ in range(2))
    pos = torch.randint(0, P, (T,), generator=g).to(I32)
    pos[0], pos[-1] = 0, P - 1
    slots = torch.randperm(R, generator=g)[:T].to(I32)
    table = bl.rope_table(P, device=dev())
    cache = torch.full((2, Hkv, R, D), 7.0, dtype=BF16, device=dev())
    qo, ko, vo = bl.qk_norm_rope(q.to(dev()), k.to(dev()), v.to(dev()), pos.to(dev()), table, q_gain=qg.to(dev()),
                                 k_gain=kg.to(dev()), slots=slots.to(dev()), k_out=cache[0].transpose(0, 1),
                                 v_out=cache[1].transpose(0, 1), halves=halves)
    _clean(bl)
    cs = table.cpu()[pos.long()]
    for name, got, x, gain in (("q", qo, q, qg), ("k", ko.cpu()[slots.long()], k, kg)):
        want, size = _rope64(x, gain, bl.RMS_EPS, cs, halves)
        _within(got, want, U8 * want.abs() + 16 * U24 * size, name)
    assert torch.equal(vo.cpu()[slots.long()], v.to(BF16))
    rest = torch.ones(R, dtype=torch.bool)
    rest[slots.long()] = False
    assert (cache.cpu()[:, :, rest] == 7.0).all(), "rows that no slot names were written"


def test_rope_without_norm_equals_the_decode_rotation(bl):
    """Bit for bit the rows that attention_decode would write, and the oracle's."""
    g = _gen(41)
    T, H, Hkv = 40, 20, 5
    q, k, v = (_rand(g, T, h, D) for h in (H, Hkv, Hkv))
    table = bl.rope_table(T, device=dev())
    qo, ko, vo = bl.qk_norm_rope(q.to(dev()), k.to(dev()), v.to(dev()),
                                 torch.arange(T, dtype=I32, device=dev()), table)
    _clean(bl)
    for t in (0, 1, 17, 39):
        for got, x, heads in ((qo, q, H), (ko, k, Hkv)):
            want = oracle.bf16_round(oracle.rope(x[t].float().numpy().reshape(-1), heads, D, t))
            np.testing.assert_array_equal(got[t].float().cpu().numpy().reshape(-1), want.reshape(-1))
    ck = torch.zeros(Hkv, T, D, dtype=BF16, device=dev())
    cv = torch.zeros_like(ck)
    for t in range(5):
        bl.attention_decode(q[t].reshape(-1).to(dev()), k[t].reshape(-1).to(dev()), v[t].reshape(-1).to(dev()), ck, cv,
                            torch.tensor([t], dtype=I32, device=dev()), H, Hkv, table=table)
    assert torch.equal(ck.transpose(0, 1)[:5], ko[:5]) and torch.equal(cv.transpose(0, 1)[:5], vo[:5])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 2500])
def test_rope_many_heads_and_padded_ones(bl, T, dtype):
    """More heads than a warp takes at once, heads that do not lie one behind
    the other, and only keys normed: equal to contiguous single calls."""
    g = _gen(T)
    H, Hkv = 64, 8
    table = bl.rope_table(64, device=dev())
    pos = (torch.arange(T, dtype=I32) % 64).to(dev())
    gain = (1 + 0.2 * torch.randn(D, generator=g)).to(dev())
    wide = torch.randn(T, H + 2 * Hkv, D + 24, generator=g).to(dtype).to(dev())
    q, k, v = wide[:, :H, 8:D + 8], wide[:, H:H + Hkv, :D], wide[:, H + Hkv:, 16:D + 16]
    a = bl.qk_norm_rope(q, k, v, pos, table, k_gain=gain)
    for x, got in ((q, a[0]), (k, a[1])):
        c = x.contiguous()
        normed = gain if x is k else None
        for h in (0, 1, x.shape[1] - 1):
            one = c[:, h:h + 1].contiguous()
            want = bl.qk_norm_rope(one, one, None, pos, table, q_gain=normed)[0]
            assert torch.equal(got[:, h:h + 1], want), h
    _clean(bl)
    assert torch.equal(a[2], v.to(BF16))
    want, size = _rope64(k.cpu(), gain.cpu(), bl.RMS_EPS, table.cpu()[pos.cpu().long()], False)
    _within(a[1], want, U8 * want.abs() + 16 * U24 * size)


def test_rope_in_place_parts_of_a_fused_projection_and_no_values(bl):
    g = _gen(43)
    T, H, Hkv = 21, 6, 2
    qkv = _rand(g, T, H + 2 * Hkv, D)
    pos = torch.arange(T, dtype=I32, device=dev())
    table = bl.rope_table(64, device=dev())
    ones = torch.ones(D, device=dev())
    for halves in (False, True):
        x = qkv.to(dev())
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        a = bl.qk_norm_rope(q, k, v, pos, table, q_gain=ones, halves=halves)
        b = bl.qk_norm_rope(q, k, None, pos, table, q_gain=ones, halves=halves)
        assert b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], v)
        bl.qk_norm_rope(q, k, v, pos, table, q_gain=ones, halves=halves, q_out=q, k_out=k, v_out=v)
        _clean(bl)
        assert torch.equal(q, a[0]) and torch.equal(k, a[1]) and torch.equal(v.cpu(), qkv[:, H + Hkv:])


def test_rope_padding_and_bad_positions_and_slots(bl):
    g = _gen(47)
    T, H, Hkv, R = 12, 4, 2, 20
    q, k, v = (_rand(g, T, h, D).to(dev()) for h in (H, Hkv, Hkv))
    table = bl.rope_table(32, device=dev())
    pos = torch.arange(T, dtype=I32)
    slots = torch.arange(T, dtype=I32) + 3

    def call(pos, slots):
        qo = torch.full((T, H, D), 7.0, dtype=BF16, device=dev())
        kv = torch.full((2, R, Hkv, D), 7.0, dtype=BF16, device=dev())
        bl.qk_norm_rope(q, k, v, pos.to(dev()), table, slots=slots.to(dev()), q_out=qo, k_out=kv[0], v_out=kv[1])
        torch.cuda.synchronize()
        return bl.last_device_status(), qo.cpu(), kv.cpu()

    st, qo, kv = call(pos, slots)
    assert st == 0
    s2 = slots.clone()
    s2[4], s2[7] = -1, -100
    st, q2, kv2 = call(pos, s2)                     # padding
    assert st == 0 and torch.equal(q2, qo)
    want = kv.clone()
    want[:, [7, 10]] = 7.0
    assert torch.equal(kv2, want)
    for p4 in (-1, 32, 2 ** 31 - 1):                # a position outside the table
        p2 = pos.clone()
        p2[4] = p4
        st, q2, kv2 = call(p2, slots)
        assert st == bl.BL_ERR_SHAPE
        want, wq = kv.clone(), qo.clone()
        want[:, 7], wq[4] = 7.0, 7.0
        assert torch.equal(kv2, want) and torch.equal(q2, wq)
    s2 = slots.clone()
    s2[4] = R                                       # a row outside the cache
    st, q2, kv2 = call(pos, s2)
    assert st == bl.BL_ERR_SHAPE and torch.equal(q2, qo)
    want = kv.clone()
    want[:, 7] = 7.0
    assert torch.equal(kv2, want)
    assert bl.last_device_status() == 0


def test_rope_rows_behind_two_to_the_31_elements(bl):
    """A cache whose last rows lie past 2^31 elements and 2^32 bytes."""
    Hkv, T = 1, 3
    R = 2 ** 31 // D + 40
    g = _gen(53)
    q, k, v = (_rand(g, T, h, D).to(dev()) for h in (2, Hkv, Hkv))
    cache = torch.empty(R, Hkv, D, dtype=BF16, device=dev())
    cache[-64:] = 7.0
    slots = torch.tensor([R - 1, R - 7, 2], dtype=I32, device=dev())
    table = bl.rope_table(8, device=dev())
    pos = torch.arange(T, dtype=I32, device=dev())
    _, ko, vo = bl.qk_norm_rope(q, k, v, pos, table)
    bl.qk_norm_rope(q, k, v, pos, table, slots=slots, k_out=cache, v_out=torch.empty(R, Hkv, D, dtype=BF16,
                                                                                     device=dev()))
    _clean(bl)
    assert torch.equal(cache[R - 1], ko[0]) and torch.equal(cache[R - 7], ko[1]) and torch.equal(cache[2], ko[2])
    assert (cache[R - 6:R - 1] == 7.0).all()
    # attention over the same far rows
    q1 = _rand(g, 1, 4, D).to(dev())
    n = 30
    cache[R - n:] = _rand(g, n, Hkv, D).to(dev())
    out = bl.attention_prefill(q1, cache, cache, _on_dev([0, 1]), _on_dev([R - n, R]))
    near = bl.attention_prefill(q1, cache[R - n:].clone(), cache[R - n:].clone(), _on_dev([0, 1]), _on_dev([0, n]))
    _clean(bl)
    want, mag = _attention_fast64(q1.cpu(), cache[R - n:].cpu(), cache[R - n:].cpu(), [0, 1], [0, n])
    tol = (U8 + 2 * 2.0 ** -12) * mag + U8 * want.abs()
    _within(out, want, tol)
    _within(near, want, tol)


# ------------------------------------------------------------------ adapters

def _adapter64(y, x, down, up, index, scale):
    """out in fp64 and the two sums of magnitudes its error bound needs."""
    want, e = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    K, r = x.shape[1], down.shape[1]
    for t, a in enumerate(index.tolist()):
        if 0 <= a < down.shape[0]:
            s = 1.0 if scale is None else float(scale[a].double())
            u = down[a].double() @ x[t].double()
            mu = down[a].double().abs() @ x[t].double().abs()
            want[t] += s * (up[a].double() @ u)
            e[t] = abs(s) * (up[a].double().abs() @ ((2.0 ** -16 + 2 * r * 2.0 ** -23) * u.abs() + K * 2.0 ** -23 * mu))
    return want, e + 4 * U24 * (y.double().abs() + want.abs())


def _check_adapter(bl, got, y, x, down, up, index, scale):
    _clean(bl)
    want, e = _adapter64(y, x, down, up, index, scale)
    _within(got, want, e + (U8 if y.dtype == BF16 else U24) * want.abs())


@pytest.mark.parametrize("T,K,N,r,n", [(1, 64, 1, 8, 1), (1, 2560, 2560, 64, 4), (5, 256, 333, 16, 3),
                                       (16, 704, 1001, 24, 16), (17, 2560, 640, 16, 5), (32, 6912, 256, 8, 32),
                                       (64, 320, 130, 128, 2), (100, 256, 257, 40, 7), (333, 512, 384, 16, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapter_add(bl, T, K, N, r, n, dtype, order):
    g = _gen(T + K + N + r)
    x, y = _rand(g, T, K), torch.randn(T, N, generator=g).to(dtype)
    down, up = _rand(g, n, r, K, s=K ** -0.5), _rand(g, n, N, r, s=r ** -0.5)
    index = torch.randint(-1, n, (T,), generator=g).to(I32)
    if T == 1:
        index[0] = n - 1
    if order == "runs":
        index = index.sort().values
    scale = 0.5 + torch.rand(n, generator=g) if order == "mixed" else None
    got = bl.adapter_add(y.to(dev()), x.to(dev()), down.to(dev()), up.to(dev()), index.to(dev()),
                         scale=None if scale is None else scale.to(dev()))
    _check_adapter(bl, got, y, x, down, up, index, scale)


@pytest.mark.parametrize("T,K,N,r,n", [(129, 2560, 264, 128, 9), (1025, 320, 1001, 64, 5), (2100, 256, 200, 16, 600),
                                       (4100, 64, 72, 8, 300), (1500, 2560, 130, 40, 20)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_adapter_of_many_alternating_requests(bl, T, K, N, r, n, dtype):
    """Tokens of many requests side by side, more adapters than are told apart
    when tokens are brought together; in place, ids that do not exist among
    them, and once more with other ids through the same graph."""
    g = _gen(T + r)
    x, y = _rand(g, T, K), torch.randn(T, N, generator=g).to(dtype)
    down, up = _rand(g, n, r, K, s=K ** -0.5), _rand(g, n, N, r, s=r ** -0.5)
    scale = 0.5 + torch.rand(n, generator=g)
    ids = [torch.randint(-1, n, (T,), generator=g).to(I32), torch.randint(-2, n, (T,), generator=g).to(I32)]
    ids[0][40:80] = n - 1
    out, index = y.to(dev()), ids[0].to(dev())
    xd, dd, ud, sd = x.to(dev()), down.to(dev()), up.to(dev()), scale.to(dev())
    bl.adapter_add(out, xd, dd, ud, index, scale=sd, out=out)
    _check_adapter(bl, out, y, x, down, up, ids[0], scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.adapter_add(out, xd, dd, ud, index, scale=sd, out=out)
    for i in (0, 1):
        index.copy_(ids[i])
        out.copy_(y)
        graph.replay()
        _check_adapter(bl, out, y, x, down, up, ids[i], scale)
    again = bl.adapter_add(y.to(dev()), xd, dd, ud, index, scale=sd)
    assert torch.equal(again, out)


def test_adapter_prompt(bl):
    g = _gen(61)
    T, K, N, r, n = 1500, 2560, 640, 16, 4
    x, y = _rand(g, T, K), _rand(g, T, N)
    down, up = _rand(g, n, r, K, s=K ** -0.5), _rand(g, n, N, r, s=r ** -0.5)
    index = torch.tensor([0] * 700 + [3] * 1 + [-1] * 299 + [2] * 500, dtype=I32)
    got = bl.adapter_add(y.to(dev()), x.to(dev()), down.to(dev()), up.to(dev()), index.to(dev()))
    _check_adapter(bl, got, y, x, down, up, index, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_adapter_none_bad_ids_pitches_and_in_place(bl, dtype):
    g = _gen(67)
    T, K, N, r, n = 37, 256, 75, 16, 3
    x, y = _rand(g, T, K + 8)[:, :K], torch.randn(T, N + 5, generator=g).to(dtype)[:, :N]
    down, up = _rand(g, n, r, K, s=K ** -0.5), _rand(g, n, N, r, s=r ** -0.5)
    big = torch.randn(T, N + 5, generator=g).to(dtype).to(dev())
    xd = torch.zeros(T, K + 8, dtype=BF16, device=dev())
    xd[:, :K] = x.to(dev())
    big[:, :N] = y.to(dev())
    rest = big[:, N:].clone()
    none = torch.full((T,), -1, dtype=I32)
    got = bl.adapter_add(big[:, :N], xd[:, :K], down.to(dev()), up.to(dev()), none.to(dev()))
    _clean(bl)
    assert torch.equal(got, big[:, :N])             # no adapter: y itself
    index = torch.randint(-1, n, (T,), generator=g).to(I32)
    index[5], index[30] = n, 2 ** 31 - 1            # adapters that do not exist
    got = bl.adapter_add(big[:, :N], xd[:, :K], down.to(dev()), up.to(dev()), index.to(dev()))
    torch.cuda.synchronize()
    assert bl.last_device_status() == bl.BL_ERR_SHAPE
    assert torch.equal(got[[5, 30]], big[[5, 30], :N])
    _check_adapter(bl, got, y, x, down, up, index, None)
    bl.adapter_add(big[:, :N], xd[:, :K], down.to(dev()), up.to(dev()), index.to(dev()), out=big[:, :N])
    torch.cuda.synchronize()
    assert bl.last_device_status() == bl.BL_ERR_SHAPE
    assert torch.equal(big[:, :N], got) and torch.equal(big[:, N:], rest)


def test_adapter_non_finite_values_stay_with_their_tokens(bl):
    """A NaN in one token's input, in an adapter that no token uses, and in one
    that other tokens use, leaves every other token as it is."""
    g = _gen(71)
    T, K, N, r, n = 20, 256, 200, 16, 4
    x, y = _rand(g, T, K), _rand(g, T, N)
    down, up = _rand(g, n, r, K, s=K ** -0.5), _rand(g, n, N, r, s=r ** -0.5)
    index = torch.tensor([0, 1, 2] * 6 + [-1, 0], dtype=I32)
    want = bl.adapter_add(y.to(dev()), x.to(dev()), down.to(dev()), up.to(dev()), index.to(dev()))
    x2, d2, u2 = x.clone(), down.clone(), up.clone()
    x2[4] = float("nan")
    x2[18] = float("inf")                           # token without an adapter
    d2[3], u2[3] = float("nan"), float("inf")       # used by nobody
    d2[2, 5], u2[2, 7] = float("inf"), float("nan")
    got = bl.adapter_add(y.to(dev()), x2.to(dev()), d2.to(dev()), u2.to(dev()), index.to(dev()))
    _clean(bl)
    rows = [t for t in range(T) if t != 4 and index[t] != 2]
    assert torch.equal(got[rows], want[rows])


def test_adapter_graph_replays_and_same_bits(bl):
    g = _gen(73)
    T, K, N, r, n = 24, 512, 300, 16, 5
    x, y = _rand(g, T, K).to(dev()), _rand(g, T, N).to(dev())
    down, up = _rand(g, n, r, K, s=K ** -0.5).to(dev()), _rand(g, n, N, r, s=r ** -0.5).to(dev())
    index = torch.zeros(T, dtype=I32, device=dev())
    out = torch.empty_like(y)
    ws = bl.adapter_workspace(T, r, dev())
    bl.adapter_add(y, x, down, up, index, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.adapter_add(y, x, down, up, index, out=out, workspace=ws)
    for _ in range(4):
        index.copy_(torch.randint(-1, n, (T,), generator=g))
        x.copy_(_rand(g, T, K))
        graph.replay()
        _clean(bl)
        assert torch.equal(out, bl.adapter_add(y, x, down, up, index))
        _check_adapter(bl, out, y.cpu(), x.cpu(), down.cpu(), up.cpu(), index.cpu(), None)


def test_adapter_writes_inside_its_buffers(bl):
    g = _gen(79)
    for T, K, N, r, n, dtype in [(33, 320, 77, 24, 3, BF16), (1, 64, 5, 8, 1, F32), (130, 256, 129, 16, 2, F32)]:
        x, y = _rand(g, T, K), torch.randn(T, N, generator=g).to(dtype)
        down, up = _rand(g, n, r, K), _rand(g, n, N, r)
        index = torch.randint(0, n, (T,), generator=g).to(I32)
        out = Guarded(T * N, dtype, dev())
        ws = Guarded(bl.adapter_workspace(T, r, dev()).numel(), torch.uint8, dev())
        bl.adapter_add(y.to(dev()), x.to(dev()), down.to(dev()), up.to(dev()), index.to(dev()), out=out.view.view(T, N),
                       workspace=ws.view)
        _check_adapter(bl, out.view.view(T, N), y, x, down, up, index, None)
        assert out.intact() and ws.intact()


# ------------------------------------------------------------------ together

def test_attention_part_of_a_layer_for_two_requests(bl):
    """Products with adapters, norm + rotation + append, attention over the
    cache: a prompt in two pieces gives what one piece gives, and its last
    token alone gives what it gave inside the prompt."""
    import synth_inputs as si
    g = _gen(83)
    hidden, H, Hkv, T = 512, 8, 2, 150
    wq, wk, wv = (bl.pack(si.weight(n * D, hidden, seed=i).to(dev())) for i, n in enumerate((H, Hkv, Hkv)))
    x = _rand(g, T, hidden).to(dev())
    down, up = _rand(g, 2, 8, hidden, s=0.04).to(dev()), _rand(g, 2, H * D, 8, s=0.3).to(dev())
    index = torch.ones(T, dtype=I32, device=dev())
    gain = torch.ones(D, dtype=BF16, device=dev())
    table = bl.rope_table(256, device=dev())
    pos = torch.arange(T, dtype=I32, device=dev())

    def piece(a, b, cache):
        q = bl.adapter_add(bl.linear(wq, x[a:b]), x[a:b], down, up, index[a:b])
        k, v = bl.linear(wk, x[a:b]), bl.linear(wv, x[a:b])
        ck, cv = (c.transpose(0, 1) for c in cache)
        q, _, _ = bl.qk_norm_rope(q.view(-1, H, D), k.view(-1, Hkv, D), v.view(-1, Hkv, D), pos[a:b], table, gain,
                                  gain, slots=pos[a:b], k_out=ck, v_out=cv)
        return q, bl.attention_prefill(q, ck, cv, _on_dev([0, b - a]), _on_dev([0, b]))

    caches = [torch.full((2, Hkv, 256, D), float("nan"), dtype=BF16, device=dev()) for _ in range(3)]
    q, whole = piece(0, T, caches[0])
    q2 = [piece(a, b, caches[1]) for a, b in ((0, 70), (70, T))]
    _clean(bl)
    # the products round per token, whichever kernel takes them: equal queries and cache rows
    assert torch.equal(torch.cat([a[0] for a in q2]), q)
    assert torch.equal(caches[0][:, :, :T], caches[1][:, :, :T])
    ck, cv = (c.transpose(0, 1)[:T].cpu() for c in caches[0])
    want, mag = _attention_fast64(q.cpu(), ck, cv, [0, T], [0, T])
    tol = (U8 + 2 * 2.0 ** -12) * mag + U8 * want.abs()
    _within(whole, want, tol)
    _within(torch.cat([a[1] for a in q2]), want, tol)
    last = bl.attention_prefill(q[-1:], *(c.transpose(0, 1) for c in caches[0]), _on_dev([0, 1]), _on_dev([0, T]))
    _within(last, want[-1:], tol[-1:])
