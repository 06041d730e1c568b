"""The attention half of one decoder layer over a prompt, in 64 bits, and how far
``Decoder.prefill`` may be from it.

The layers here have a feed-forward block of zero weights and small streams, so
what a token's stream gains is the o product of its attention and nothing
drowns it.  Queries, keys and values come from the oracle bit for bit (RMSNorm +
quantisation, products, rotation).  For token t with attention a (fp64, sums of
magnitudes g = sum_j w_j |V_j|), K values and the dequantised o weights W:

  kernel's attention   |a' - a| <= e = (2^-8 + 2 * 2^-12) g + 2^-8 |a|
                       (a weight's rounding and its exponential; the output's)
  quantised            one step is absmax(a') / 127, off by at most half of it
  product              exact integers, so |W (q - a)| <= s ||q - a||, s = W's
                       largest singular value
  stream               bf16(x + y): 2^-8 of it (the fp32 steps: 2^-20 of it)

  ||gain - W a|| <= s (||e|| + sqrt(K) / 2 * (max |a| + max e) / 127)
                    + (2^-8 + 2^-20) (||x + W a|| + the first term)
"""
import numpy as np
import torch

import oracle
import synth_inputs as si
from parity_helpers import oracle_weight

D = 128
MISTAKES = ("one key more", "one key less", "queries not rotated", "keys not rotated", "queries a position late",
            "equal weights", "heads crossed", "twice the scale", "pieces forget the past")


def config(hidden, heads, kv_heads, max_seq=80, layers=1):
    from bit_ternary_weight_b200.decoder import DecoderConfig
    return DecoderConfig(hidden=hidden, heads=heads, kv_heads=kv_heads, ffn=256, layers=layers, max_seq=max_seq)


def weights(cfg, seed):
    """Scores of a standard deviation of one to three, so that weights are
    neither equal nor one."""
    shapes = {"q": (cfg.heads * D, cfg.hidden), "k": (cfg.kv_heads * D, cfg.hidden), "v": (cfg.kv_heads * D, cfg.hidden),
              "o": (cfg.hidden, cfg.heads * D), "gate": (cfg.ffn, cfg.hidden), "up": (cfg.ffn, cfg.hidden),
              "down": (cfg.hidden, cfg.ffn)}
    std = {"q": 0.1 * (512 / cfg.hidden) ** 0.5, "k": 0.1 * (512 / cfg.hidden) ** 0.5, "down": 0.0}
    w = {n: si.weight(N, K, seed=seed * 100 + j, std=std.get(n, 0.02)) for j, (n, (N, K)) in enumerate(shapes.items())}
    for j, name in enumerate(("g_attn", "g_ffn")):
        w[name] = (1.0 + 0.1 * si.activations(1, cfg.hidden, seed=seed * 7 + j, outliers=False,
                                              dtype=torch.float32)[0]).to(torch.bfloat16)
    return w


def prompt(cfg, T, seed):
    return (si.activations(T, cfg.hidden, seed=seed).float() * 2.0 ** -6).to(torch.bfloat16)


class Layer:
    """Queries and keys (before and after rotation) and values of a prompt."""

    def __init__(self, cfg, w, x):
        self.cfg, self.x = cfg, x.double().numpy()
        T, H, Hkv = x.shape[0], cfg.heads, cfg.kv_heads
        gain, xs = w["g_attn"].float().numpy(), x.float().numpy()

        def product(name, n):
            g, codes, _ = oracle_weight(w[name])
            y = np.stack([oracle._linear32(row, codes, g, gain, cfg.eps) for row in xs])
            return oracle.bf16_round(y).reshape(T, n, D)

        self.q, self.k, self.v = product("q", H), product("k", Hkv), product("v", Hkv).astype(np.float64)
        g, codes, _ = oracle_weight(w["o"])
        self.o = float(g) * codes.astype(np.float64)
        self.s = float(torch.linalg.matrix_norm(torch.from_numpy(self.o), 2))

    def _rotated(self, a, shift=0):
        rows = [oracle.bf16_round(oracle.rope(r.reshape(-1), r.shape[0], D, t + shift, self.cfg.rope_base))
                for t, r in enumerate(a)]
        return np.stack(rows).reshape(a.shape)

    def gain(self, mistake=None, cut=0):
        """(W a [T, hidden], bound on the 2-norm of each row's difference)."""
        T, H, Hkv = self.q.shape[0], self.cfg.heads, self.cfg.kv_heads
        q = self.q if mistake == "queries not rotated" else self._rotated(self.q, mistake == "queries a position late")
        k = self.k if mistake == "keys not rotated" else self._rotated(self.k)
        head = np.arange(H) % Hkv if mistake == "heads crossed" else np.arange(H) // (H // Hkv)
        s = np.einsum("thd,jhd->htj", q.astype(np.float64), k.astype(np.float64)[:, head]) / D ** 0.5
        if mistake == "equal weights":
            s[:] = 0.0
        if mistake == "twice the scale":
            s *= 2.0
        seen = np.arange(T) + 1 + {"one key more": 1, "one key less": -1}.get(mistake, 0)
        if mistake == "pieces forget the past":
            seen = np.where(np.arange(T) >= cut, seen - cut, seen)
        mask = np.arange(T)[None] < seen[:, None]
        p = np.where(mask, np.exp(s - s.max(-1, keepdims=True)), 0.0)
        p /= np.maximum(p.sum(-1, keepdims=True), 1e-300)
        v = self.v[:, head]
        a = np.einsum("htj,jhd->thd", p, v).reshape(T, -1)
        g = np.einsum("htj,jhd->thd", p, np.abs(v)).reshape(T, -1)
        e = (2.0 ** -8 + 2 * 2.0 ** -12) * g + 2.0 ** -8 * np.abs(a)
        step = (np.abs(a).max(-1) + e.max(-1)) / 127
        tol = self.s * (np.linalg.norm(e, axis=-1) + 0.5 * a.shape[1] ** 0.5 * step)
        y = a @ self.o.T
        tol += (2.0 ** -8 + 2.0 ** -20) * (np.linalg.norm(self.x + y, axis=-1) + tol)
        return y, tol
