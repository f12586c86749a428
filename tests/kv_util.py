"""Ragged batches over the 8-bit paged cache for the tests: numpy inputs, a
random page table, and the comparison with the float64 oracle."""
import numpy as np
import torch

import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq

DEV = "cuda"


def bf16(x):
    """(bf16 CUDA tensor, its values in float64)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


class Batch:
    """q_lens new rows and kv_lens tokens of each sequence; `spare` pages of
    nobody, `behind` rows behind the last sequence."""

    def __init__(self, q_lens, kv_lens, H, d, P, seed=0, spare=3, behind=0, v_spread=0.0):
        self.g = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.H, self.d, self.P = q_lens, kv_lens, H, d, P
        pages = [-(-n // P) for n in kv_lens]
        self.pages = sum(pages) + spare
        ids = self.g.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(kv_lens), max(pages + [1]) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.cu = np.cumsum([0] + list(q_lens)).astype(np.int32)
        self.N = int(self.cu[-1]) + behind
        self.kv_len = np.asarray(kv_lens, np.int32)
        shape = (self.pages, H, P, d)
        self.kc, self.vc = (self.g.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        self.ks = (self.g.uniform(0.5, 2.0, shape[:2]) / 64).astype(np.float32)
        self.vs = (self.g.uniform(0.5, 2.0, shape[:2]) * np.exp2(self.g.uniform(-v_spread, v_spread, shape[:2])) / 64).astype(np.float32)

    def to_gpu(self):
        self.cache = rq.KvCache(*(torch.from_numpy(x.copy()).to(DEV) for x in (self.kc, self.vc, self.ks, self.vs)))
        self.t_cu, self.t_len, self.t_table = (torch.from_numpy(x).to(DEV) for x in (self.cu, self.kv_len, self.table))
        return self


def workspace(cache, Hq, N, max_q=None):
    # filled with NaN: nothing of it may be read before it is written
    n = rq.respin_kv_attention_workspace(cache, Hq, N, max_q)
    return torch.full(((n + 3) // 4,), float("nan"), device=DEV).view(torch.uint8)


def attend(bt, Hq, *, causal=True, window=0, scale=None, use_cu=True, max_q="max", q=None, seed=1, q_gain=1.0):
    """Run respin_kv_attention on the batch and check it against the oracle.

    Tolerance, from the kernel's roundings (half a step each): the bf16 output
    2^-8 of itself; each weight's fp16 rounding 2^-11 of its part of
    sum w |v|; its fp32 exponent, of size up to 2^8, 2^-16 (16 half steps of
    2^-24 at 2^8 is 2^-12 in the worst case, reached only by weights of 2^-8
    of the row's sum: 2^-16 beside the row); fp16's floor, 2^-25 (half of
    its smallest step) beside a largest weight of 2^2 at least, for every token: n 2^-27 of the largest."""
    g = np.random.default_rng(seed)
    d = bt.d
    scale = d ** -0.5 if scale is None else scale
    if q is None:
        q = g.standard_normal((bt.N, Hq, d)) * q_gain
    tq, q64 = bf16(q)
    out = torch.full((bt.N, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((bt.N, Hq), 7.0, dtype=torch.float32, device=DEV)
    mq = max(bt.q_lens) if max_q == "max" else max_q
    ws = workspace(bt.cache, Hq, bt.N, mq)
    rq.respin_kv_attention(bt.cache, tq, bt.t_len, bt.t_table, out, ws, cu=bt.t_cu if use_cu else None,
                           max_q=mq, causal=causal, window=window, scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert rq.respin_device_status() == 0
    n = int(bt.cu[-1])
    ref, rl, spread, top = AO.attention(q64[:n], bt.kc, bt.vc, bt.ks, bt.vs, bt.cu, bt.kv_len, bt.table, bt.P,
                                        scale=scale, causal=causal, window=window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[n:] == 7).all() and (gl[n:] == 7).all()      # rows behind the last sequence
    got, gl = got[:n], gl[:n]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -16) * spread + max(bt.kv_lens) * 2.0 ** -27 * top[..., None]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], bad.mean())
    empty = np.isinf(rl)
    assert (gl[empty] == -np.inf).all() and (got[empty] == 0).all()
    # lse: an exponent of size up to 2^8 in fp32, and the sum
    gl, rl = gl[~empty], rl[~empty]
    bad = ~(np.abs(gl - rl) <= 2.0 ** -15 + 2.0 ** -22 * np.abs(rl))
    assert not bad.any(), (gl[bad][:5], rl[bad][:5], bad.mean())
    return out, lse
